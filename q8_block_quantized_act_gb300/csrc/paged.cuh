// paged.cuh -- a batch of sequences over a paged key/value cache (q8act_paged_kv), as its kernels
// read it.  Everything that comes from device memory (starts, lens, page ids) is clamped or checked
// here, so no value in it leads to an access out of bounds or a loop without end.
#pragma once

#include "common.cuh"

namespace q8 {

struct Paged {
    const int32_t *__restrict__ table;
    const int32_t *__restrict__ starts;
    const int32_t *__restrict__ lens;
    int64_t table_ld, page_stride, pages;
    int seqs, width, page_shift, heads, m;    // heads: of keys and values; m: rows that the call was given
    int capacity;                             // positions that the table can hold
};

inline Paged paged_of(const q8act_paged_kv &kv, int64_t m)
{
    Paged p;
    p.table = kv.table;
    p.starts = kv.starts;
    p.lens = kv.lens;
    p.table_ld = kv.table_ld;
    p.page_stride = kv.page_stride;
    p.pages = kv.pages;
    p.seqs = kv.seqs;
    p.width = kv.table_width;
    p.page_shift = __builtin_ctz((unsigned)kv.page_size);
    p.heads = kv.heads;
    p.m = (int)m;
    p.capacity = kv.table_width << p.page_shift;
    return p;
}

// A sequence's part of the batch: its new tokens are rows row0 .. row0 + n - 1 at positions pos0,
// pos0 + 1, ...; the cache holds positions 0 .. end - 1 (pos0 < 0: more new tokens than positions).
struct Seq {
    int row0, n, pos0, end;
};

__device__ __forceinline__ Seq seq_of(const Paged &p, int b)
{
    const int s0 = min(max(__ldg(p.starts + b), 0), p.m), s1 = min(max(__ldg(p.starts + b + 1), s0), p.m);
    const int len = max(__ldg(p.lens + b), 0);
    Seq s;
    s.row0 = s0;
    s.n = s1 - s0;
    s.pos0 = len - s.n;
    s.end = min(len, p.capacity);
    return s;
}

// The page of a sequence's table entry, or -1 where the table or the cache does not have it.
__device__ __forceinline__ int64_t page_of(const Paged &p, int b, int entry)
{
    if (entry >= p.width) return -1;
    const int64_t id = __ldg(p.table + b * p.table_ld + entry);
    return id >= 0 && id < p.pages ? id : -1;
}

}  // namespace q8
