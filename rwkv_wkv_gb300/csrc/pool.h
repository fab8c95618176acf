// The pool object behind the C-ABI's opaque handle, shared by the entry points
// of capi.cpp, gdn_capi.cpp and ssm_capi.cpp.
#pragma once

#include "wkv7.h"

#include <mutex>
#include <vector>

#include "wkv7_internal.h"

namespace wkv7 {

// Host-side id table: a LIFO free list plus an "in use" flag per id.
struct IdTable {
    std::vector<int32_t> free_list;
    std::vector<uint8_t> used;

    void init(int32_t n) {
        used.assign(static_cast<size_t>(n), 0);
        free_list.resize(static_cast<size_t>(n));
        for (int32_t i = 0; i < n; ++i) free_list[static_cast<size_t>(i)] = n - 1 - i;
    }
    int32_t size() const { return static_cast<int32_t>(used.size()); }
    int32_t n_free() const { return static_cast<int32_t>(free_list.size()); }

    wkv7_status alloc(int32_t n, int32_t *out) {
        if (n < 0 || (n > 0 && !out)) return WKV7_ERR_INVALID_ARG;
        if (n > n_free()) return WKV7_ERR_POOL_FULL;
        for (int32_t i = 0; i < n; ++i) {
            int32_t id = free_list.back();
            free_list.pop_back();
            used[static_cast<size_t>(id)] = 1;
            out[i] = id;
        }
        return WKV7_OK;
    }

    wkv7_status release(int32_t n, const int32_t *ids) {
        if (n < 0 || (n > 0 && !ids)) return WKV7_ERR_INVALID_ARG;
        std::vector<uint8_t> seen(used.size(), 0);
        for (int32_t i = 0; i < n; ++i) {  // validate everything first
            int32_t id = ids[i];
            if (id < 0 || id >= size() || !used[static_cast<size_t>(id)]) return WKV7_ERR_BAD_SLOT;
            if (seen[static_cast<size_t>(id)]) return WKV7_ERR_DUP_SLOT;
            seen[static_cast<size_t>(id)] = 1;
        }
        for (int32_t i = 0; i < n; ++i) {
            used[static_cast<size_t>(ids[i])] = 0;
            free_list.push_back(ids[i]);
        }
        return WKV7_OK;
    }
};

// Count a call's launches and turn a CUDA error into the call's status.
wkv7_status cuda_status(const char *what, cudaError_t e, int launches);

// Lay a pool whose description has been checked over its buffer (the caller's,
// or one allocated here) and register it: slots of slot_bytes bytes each.
wkv7_status lay_out_pool(wkv7_pool *p, size_t slot_bytes, size_t need, wkv7_pool **out);
// Bytes that the tails of a short convolution add to a slot.
size_t conv_bytes(const wkv7_conv_desc &c, int32_t n_layers);
bool conv_desc_valid(const wkv7_conv_desc &c);
// Bytes of a pool: header, slots, snapshots, id bitmap.
size_t pool_bytes(const wkv7_pool_desc *d, size_t slot_bytes);

}  // namespace wkv7

struct wkv7_pool {
    wkv7_pool_desc desc{};
    char *base = nullptr;
    bool owns = false;
    int32_t *status = nullptr;
    float *states = nullptr;
    float *snaps = nullptr;
    uint32_t *marks = nullptr;  // id-validation bitmap (scratch of wkv7_validate_ids)
    long long slot_floats = 0;  // slot bytes / 4: the unit of the byte-copy verbs
    long long slot_entries = 0; // slot bytes / bytes of a state entry: from one slot's states to the next's
    bool state_bf16 = false;
    bool out_bf16 = false;  // o written in bf16
    long long head_elems = wkv7::kHeadFloats;  // state entries of one head
    bool gdn = false;       // a gated-delta-rule pool (wkv7_gdn_pool_create): heads as in `gdn_desc`
    wkv7_gdn_pool_desc gdn_desc{};
    bool ssm = false;       // a pool of scan states (wkv7_ssm_pool_create)
    wkv7_ssm_pool_desc ssm_desc{};
    wkv7_conv_desc conv{};  // the tails behind a slot's states (channels == 0: none) ...
    size_t conv_off = 0;    // ... from this byte of the slot on
    bool wkv() const { return !gdn && !ssm; }
    std::mutex mu;
    wkv7::IdTable slots;
    wkv7::IdTable snapshots;
};
