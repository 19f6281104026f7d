// Device-side helpers of the key-value cache: where a token lies.
#pragma once

#include "attention_kernels.hpp"
#include "ct_device.hpp"

namespace ct {

typedef unsigned int uint4v __attribute__((ext_vector_type(4)));

__device__ __forceinline__ int clampi(int v, int lo, int hi) { return v < lo ? lo : v > hi ? hi : v; }

// A sequence's new tokens: rows [first, first + count) of the call's tokens.
// Every count is held to the call's tokens, whatever starts hold.
struct Span {
    int first, count;
};

__device__ __forceinline__ Span span_of(const KvBatch& b, int seq) {
    if (!b.starts) return {seq * b.even, b.even};
    const int s = clampi(b.starts[seq], 0, b.tokens), e = clampi(b.starts[seq + 1], s, b.tokens);
    return {s, e - s};
}

// Tokens in the cache: at most 2^30, so that places and distances stay in 32 bits.
__device__ __forceinline__ int length_of(const KvBatch& b, int seq) { return clampi(b.lens[seq], 0, 1 << 30); }

// The sequence of a token; -1 outside of all.
__device__ __forceinline__ int sequence_of(const KvBatch& b, int token) {
    if (!b.starts) return token / b.even;
    // the last start that is at most `token`
    int lo = -1, hi = b.sequences + 1;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (b.starts[mid] <= token) lo = mid;
        else hi = mid;
    }
    return lo >= 0 && lo < b.sequences ? lo : -1;
}

// A place's page in the sequence, and the place in it.
struct Place {
    int index, in;
};

__device__ __forceinline__ Place place_of(const KvPages& c, int pos) {
    const int i = (int)(((unsigned long long)(unsigned)pos * c.magic) >> c.shift);
    return {i, pos - i * c.page};
}

// The page that the table names; not checked against the pool.
__device__ __forceinline__ int page_of(const KvBatch& b, int seq, int index) {
    return b.table ? b.table[(long long)seq * b.ldt + index] : seq;
}

__device__ __forceinline__ uint16_t to_half(float f, int dt) {
    return dt == DT_BF16 ? __builtin_bit_cast(uint16_t, (__bf16)f) : __builtin_bit_cast(uint16_t, (_Float16)f);
}

}  // namespace ct
