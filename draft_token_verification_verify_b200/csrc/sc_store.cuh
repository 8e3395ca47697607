// Writing the 4-bit cache and reading it back.
//
// K_append quantises the kept rows behind each sequence's length; K_read
// expands a range of every sequence.  In both a group of D / 4 lanes (a warp at
// D = 128, half a warp at D = 64) takes one (sequence, 8 tokens of a block,
// head) and each lane 4 dims, so that the word of 8 tokens of a value row
// (values are stored dim by dim) is built, or taken apart, within one lane.
// Heads are the fastest index of the groups: neighbours read, or write, whole
// token rows.  Both are bound by the bytes they move; nothing is read twice.
#pragma once

#include "sc_common.cuh"

namespace sv {

constexpr int SC_STORE_NT = 128;

struct AppendParams {
    const void* k;
    const void* v;
    long long stride;  // elements between tokens
    int B, n;
    const int32_t* n_accepted;  // or null
    const int32_t* nodes;       // or null
    int nodes_stride;
    int32_t* out_lens;  // null when a later kernel advances the lengths in place
    int ngrp;           // groups of 8 positions a sequence's new rows can touch
};

struct ReadParams {
    const int32_t* first;  // or null
    void* out_k;
    void* out_v;
    int B, n;
    int ngrp;
};

// min of bf16 / fp16 pairs, NaN if either is.
template <int DT>
__device__ __forceinline__ uint32_t sc_min2(uint32_t a, uint32_t b) {
    uint32_t d;
    if constexpr (DT == 0)
        asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    else
        asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// The rows sequence b keeps and whether its call is sound (all lanes alike).
__device__ __forceinline__ bool sc_kept(const CacheView& c, const AppendParams& P, int b, int* len, int* count) {
    *len = c.lens[b];
    int m = P.n;
    if (P.n_accepted) {
        const int a = P.n_accepted[b];
        m = a < 0 ? 0 : (a >= P.n ? -1 : a + 1);  // more rows than there are: a data error
    }
    *count = m;
    return *len >= 0 && m >= 0 && static_cast<long long>(*len) + m <= sc_capacity(c);
}

__device__ __forceinline__ int sc_node(const AppendParams& P, int b, int row) {
    return (row == 0 || !P.nodes) ? row : P.nodes[static_cast<size_t>(b) * P.nodes_stride + row - 1];
}

// The new length of sequence b, by `lanes` lanes of a group (lane l, mask m):
// -1 where a page or a node it needs is out of range.
template <int LPI>
__device__ __forceinline__ int sc_new_len(const CacheView& c, const AppendParams& P, int b, int l, unsigned mask) {
    int len, count;
    const bool sound = sc_kept(c, P, b, &len, &count);
    if (len < 0) return len;
    int bad = !sound;
    if (sound && count > 0) {
        for (int p = (len >> c.log2_page) + l; p <= ((len + count - 1) >> c.log2_page); p += LPI) {
            const int id = c.table[static_cast<size_t>(b) * c.max_pages + p];
            bad |= id < 0 || id >= c.num_pages;
        }
        for (int r = l; r < count; r += LPI) {
            const int node = sc_node(P, b, r);
            bad |= node < 0 || node >= P.n;
        }
    }
    return __any_sync(mask, bad) ? -1 : len + count;
}

// One step of a reduce-scatter over N registers: lanes whose bit `O` is set
// keep the upper half.
template <int DT, int N, int O>
__device__ __forceinline__ void sc_fold(uint32_t (&x)[16], int l, unsigned mask) {
    const bool up = (l & O) != 0;
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        const uint32_t keep = up ? x[i + N / 2] : x[i];
        const uint32_t give = up ? x[i] : x[i + N / 2];
        x[i] = sc_min2<DT>(keep, __shfl_xor_sync(mask, give, O));
    }
}

// The codes of 4 elements as floats: (x - zero) / scale rounded to the nearest
// whole number, ties to even, as the exact fp32 quotient decides.  The product
// with the reciprocal is within 1e-5 of that quotient (which stays below 15.1
// while the scale is a normal number); where it comes that close to a half, or
// the reciprocal is of no use (NaN), the quotients are formed.
__device__ __forceinline__ float sc_code(float d, float scale) {
    const float c = scale > 0.f ? fminf(rintf(__fdiv_rn(d, scale)), 15.f) : 0.f;
    return c >= 0.f ? c : 0.f;
}
__device__ __forceinline__ void sc_codes4(uint64_t x01, uint64_t x23, float zero, float scale, float inv,
                                          uint64_t& c01, uint64_t& c23) {
    const uint64_t nz = f2_pack(-zero, -zero), i2 = f2_pack(inv, inv);
    const uint64_t up = f2_pack(12582912.f, 12582912.f), down = f2_pack(-12582912.f, -12582912.f);
    const uint64_t d01 = f2_add(x01, nz), d23 = f2_add(x23, nz);
    const uint64_t q01 = f2_mul(d01, i2), q23 = f2_mul(d23, i2);
    c01 = f2_add(f2_add(q01, up), down);
    c23 = f2_add(f2_add(q23, up), down);
    float a, b, c, d, e0, e1, e2, e3;
    f2_unpack(c01, a, b);
    f2_unpack(c23, c, d);
    f2_unpack(q01, e0, e1);
    f2_unpack(q23, e2, e3);
    const float off = fmaxf(fmaxf(fabsf(e0 - a), fabsf(e1 - b)), fmaxf(fabsf(e2 - c), fabsf(e3 - d)));
    if (off >= 0.49998f || inv != inv) {
        f2_unpack(d01, a, b);
        f2_unpack(d23, c, d);
        c01 = f2_pack(sc_code(a, scale), sc_code(b, scale));
        c23 = f2_pack(sc_code(c, scale), sc_code(d, scale));
    }
}

// Low 16 bits: a whole number below 2^16 held in a float.
__device__ __forceinline__ uint32_t sc_bits(float c) { return __float_as_uint(c + 8388608.f); }

template <int DT, int D>
__global__ void __launch_bounds__(SC_STORE_NT) sc_append_kernel(CacheView c, AppendParams P) {
    using Ty = SC<DT>;
    constexpr int LPI = D / 4;
    const int lane = threadIdx.x & 31, l = lane % LPI;
    const unsigned mask = LPI == 32 ? 0xffffffffu : 0xffffu << (lane & 16);
    const long long item = (static_cast<long long>(blockIdx.x) * SC_STORE_NT + threadIdx.x) / LPI;
    const int h = static_cast<int>(item % c.kv_heads);
    const long long bj = item / c.kv_heads;
    const int j = static_cast<int>(bj % P.ngrp);
    const long long bl = bj / P.ngrp;
    if (bl >= P.B) return;
    const int b = static_cast<int>(bl);
    if (P.out_lens && h == 0 && j == 0) {
        const int nl = sc_new_len<LPI>(c, P, b, l, mask);
        if (l == 0) P.out_lens[b] = nl;
    }
    int len, count;
    if (!sc_kept(c, P, b, &len, &count) || count == 0) return;
    const int T = c.block;
    const int p0 = ((len >> 3) + j) << 3;  // first position of the group
    if (p0 >= len + count) return;
    const int t0 = p0 & ~(T - 1);          // and of its block
    const int from = len > t0 ? len - t0 : 0;                     // tokens of the block written:
    const int to = len + count - t0 < T ? len + count - t0 : T;  // [from, to)
    const int id = c.table[static_cast<size_t>(b) * c.max_pages + (t0 >> c.log2_page)];
    if (id < 0 || id >= c.num_pages) return;
    unsigned char* blkp = sc_block_ptr<D>(c, id, h, (t0 & (c.page_size - 1)) >> c.log2_block);
    unsigned char* vblk = blkp + sc_half_bytes<D>(T);

    const int g = (p0 - t0) >> 3;
    // 8 tokens: 4 dims of each, keys and values
    uint2 raw[16];
    uint32_t have = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int t = g * 8 + i;
        raw[i] = raw[8 + i] = make_uint2(0u, 0u);
        if (t >= from && t < to) {
            const int node = sc_node(P, b, t0 + t - len);
            if (node >= 0 && node < P.n) {
                have |= 1u << i;
                const size_t o = (static_cast<size_t>(b) * P.n + node) * static_cast<size_t>(P.stride) +
                                 static_cast<size_t>(h) * D + 4 * l;
                raw[i] = *reinterpret_cast<const uint2*>(static_cast<const typename Ty::T*>(P.k) + o);
                raw[8 + i] = *reinterpret_cast<const uint2*>(static_cast<const typename Ty::T*>(P.v) + o);
            }
        }
    }
    // each row's {min, -max}: within the lane, then a reduce-scatter of the
    // 16 rows over the lanes (15 exchanges of one register, and one more at
    // 32 lanes, in place of 5 steps for each row and side)
    uint32_t x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const uint32_t lo = sc_min2<DT>(raw[i].x, raw[i].y);
        const uint32_t hi = sc_min2<DT>(raw[i].x ^ 0x80008000u, raw[i].y ^ 0x80008000u);
        x[i] = sc_min2<DT>(__byte_perm(lo, hi, 0x5410), __byte_perm(lo, hi, 0x7632));
    }
    sc_fold<DT, 16, 1>(x, l, mask);
    sc_fold<DT, 8, 2>(x, l, mask);
    sc_fold<DT, 4, 4>(x, l, mask);
    sc_fold<DT, 2, 8>(x, l, mask);
    if (LPI == 32) x[0] = sc_min2<DT>(x[0], __shfl_xor_sync(mask, x[0], 16));
    // lane l holds row 8 b0 + 4 b1 + 2 b2 + b3 (b the bits of l): its (scale, zero), and what a
    // difference from zero is multiplied by (NaN: it is divided, see sc_codes4)
    uint32_t par;
    float inv;
    {
        const float mn = Ty::lo(x[0]), mx = -Ty::hi(x[0]);
        const float sc = Ty::round(__fdiv_rn(__fsub_rn(mx, mn), 15.f));
        const bool fine = fabsf(mn) < __builtin_huge_valf() && fabsf(mx) < __builtin_huge_valf() &&
                          fabsf(sc) < __builtin_huge_valf();
        par = fine ? Ty::pack(sc, mn) : 0x00007fffu;  // a NaN in either type
        inv = fine && sc >= (DT == 0 ? 1e-30f : 6.2e-5f) ? __fdividef(1.f, sc) : __int_as_float(0x7fffffff);
    }
    uint64_t vacc[2][2];  // dims {0, 1} and {2, 3} of the lane: the even and the odd tokens' codes
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int src = ((i >> 3) & 1) | ((i >> 1) & 2) | ((i << 1) & 4) | ((i << 3) & 8);
        const uint32_t p = __shfl_sync(mask, par, src, LPI);
        const float iv = __shfl_sync(mask, inv, src, LPI);
        uint64_t c01, c23;
        sc_codes4(f2_pack(Ty::lo(raw[i].x), Ty::hi(raw[i].x)), f2_pack(Ty::lo(raw[i].y), Ty::hi(raw[i].y)), Ty::hi(p),
                  Ty::lo(p), iv, c01, c23);
        const int t = g * 8 + (i & 7);
        const bool mine = (have >> (i & 7)) & 1u;
        if (i < 8) {
            // a key row's word w: dims 8w.. from lanes 2w (low byte of each half) and 2w+1
            float lo, hi;
            f2_unpack(f2_fma(f2_pack(16.f, 16.f), c23, c01), lo, hi);
            uint32_t w = __byte_perm(sc_bits(lo), sc_bits(hi), (l & 1) ? 0x4707 : 0x7470) &
                         ((l & 1) ? 0xFF00FF00u : 0x00FF00FFu);
            w |= __shfl_xor_sync(mask, w, 1);
            if (mine) {
                if ((l & 1) == 0) *reinterpret_cast<uint32_t*>(blkp + t * (D / 2) + (l >> 1) * 4) = w;
                if (l == 1) *reinterpret_cast<uint32_t*>(blkp + T * (D / 2) + t * 4) = p;
            }
        } else {
            const int e = i & 1, m = (i & 7) >> 1;  // token 2m + e: bits 16e + 4m
            const float f = m == 1 ? 16.f : m == 2 ? 256.f : 4096.f;
            vacc[0][e] = m == 0 ? c01 : f2_fma(f2_pack(f, f), c01, vacc[0][e]);
            vacc[1][e] = m == 0 ? c23 : f2_fma(f2_pack(f, f), c23, vacc[1][e]);
            if (l == 0 && mine) *reinterpret_cast<uint32_t*>(vblk + T * (D / 2) + t * 4) = p;
        }
    }
    // tokens of the group that are not written keep their codes
    uint32_t keep = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (!((have >> i) & 1u)) keep |= 0xFu << (16 * (i & 1) + 4 * (i >> 1));
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        float e0, e1, o0, o1;
        f2_unpack(vacc[q][0], e0, e1);
        f2_unpack(vacc[q][1], o0, o1);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            uint32_t w = __byte_perm(sc_bits(k ? e1 : e0), sc_bits(k ? o1 : o0), 0x5410);
            uint32_t* dst = reinterpret_cast<uint32_t*>(vblk + (4 * l + 2 * q + k) * (T / 2) + g * 4);
            if (keep) w = (w & ~keep) | (*dst & keep);
            *dst = w;
        }
    }
}

// The lengths advanced in place, after every block has been written.
__global__ void __launch_bounds__(SC_STORE_NT) sc_advance_kernel(CacheView c, AppendParams P, int32_t* out_lens) {
    pdl_wait_primary();
    const int b = blockIdx.x * (SC_STORE_NT / 32) + (threadIdx.x >> 5);
    if (b >= P.B) return;
    const int l = threadIdx.x & 31;
    const int nl = sc_new_len<32>(c, P, b, l, 0xffffffffu);
    if (l == 0) out_lens[b] = nl;
}

// Four codes at bit 0 (lane even) or 8 (odd) of a key word as floats.
__device__ __forceinline__ float sc_code_f(uint32_t w, int shift) {
    return __uint_as_float(((w >> shift) & 15u) | 0x4B000000u) - 8388608.f;
}

template <int DT, int D>
__global__ void __launch_bounds__(SC_STORE_NT) sc_read_kernel(CacheView c, ReadParams P) {
    using Ty = SC<DT>;
    constexpr int LPI = D / 4;
    const int l = threadIdx.x % LPI;
    const long long item = (static_cast<long long>(blockIdx.x) * SC_STORE_NT + threadIdx.x) / LPI;
    const int h = static_cast<int>(item % c.kv_heads);
    const long long bj = item / c.kv_heads;
    const int j = static_cast<int>(bj % P.ngrp);
    const long long bl = bj / P.ngrp;
    if (bl >= P.B) return;
    const int b = static_cast<int>(bl);
    const int len = c.lens[b];
    const long long first = P.first ? P.first[b] : 0;
    const int T = c.block;
    const long long p0 = ((first >> 3) + j) * 8;  // first position of the group, may be negative
    if (p0 >= first + P.n) return;
    const long long t0 = p0 & ~static_cast<long long>(T - 1);  // and of its block
    const int from = static_cast<int>(first > t0 ? first - t0 : 0);
    const int to = static_cast<int>(first + P.n - t0 < T ? first + P.n - t0 : T);
    const unsigned char* blkp = nullptr;
    bool bad = false;
    if (t0 >= 0 && t0 < len) {
        bad = t0 >= sc_capacity(c);
        if (!bad) {
            const int id = c.table[static_cast<size_t>(b) * c.max_pages + (t0 >> c.log2_page)];
            bad = id < 0 || id >= c.num_pages;
            if (!bad)
                blkp = sc_block_ptr<D>(c, id, h, (static_cast<int>(t0) & (c.page_size - 1)) >> c.log2_block);
        }
    }
    const unsigned char* vblk = blkp ? blkp + sc_half_bytes<D>(T) : nullptr;
    typename Ty::T* ok = static_cast<typename Ty::T*>(P.out_k);
    typename Ty::T* ov = static_cast<typename Ty::T*>(P.out_v);
    const int g = static_cast<int>(p0 - t0) >> 3;
    {
        uint32_t vw[4] = {0u, 0u, 0u, 0u}, kw[8];
        uint32_t kp[8], vp[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            kw[i] = kp[i] = vp[i] = 0u;
            const int t = g * 8 + i;
            if (blkp && t >= from && t < to) {
                if (ok) {
                    kw[i] = *reinterpret_cast<const uint32_t*>(blkp + t * (D / 2) + (l >> 1) * 4);
                    kp[i] = *reinterpret_cast<const uint32_t*>(blkp + T * (D / 2) + t * 4);
                }
                if (ov) vp[i] = *reinterpret_cast<const uint32_t*>(vblk + T * (D / 2) + t * 4);
            }
        }
        if (blkp && ov) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                vw[q] = *reinterpret_cast<const uint32_t*>(vblk + (4 * l + q) * (T / 2) + g * 4);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int t = g * 8 + i;
            if (t < from || t >= to) continue;
            const long long pos = t0 + t;
            const size_t o = ((static_cast<size_t>(b) * P.n + static_cast<size_t>(pos - first)) * c.kv_heads + h) *
                                 static_cast<size_t>(D) + 4 * l;
            const bool in = pos >= 0 && pos < len;
            if (ok) {
                uint2 w = make_uint2(0u, 0u);
                if (in && bad) w = make_uint2(0x7fff7fffu, 0x7fff7fffu);
                if (in && !bad) {
                    const float s = Ty::lo(kp[i]), z = Ty::hi(kp[i]);
                    const uint32_t x = kw[i] >> (8 * (l & 1));
                    w.x = Ty::pack(fmaf(s, sc_code_f(x, 0), z), fmaf(s, sc_code_f(x, 16), z));
                    w.y = Ty::pack(fmaf(s, sc_code_f(x, 4), z), fmaf(s, sc_code_f(x, 20), z));
                }
                *reinterpret_cast<uint2*>(ok + o) = w;
            }
            if (ov) {
                uint2 w = make_uint2(0u, 0u);
                if (in && bad) w = make_uint2(0x7fff7fffu, 0x7fff7fffu);
                if (in && !bad) {
                    const float s = Ty::lo(vp[i]), z = Ty::hi(vp[i]);
                    const int sh = 16 * (i & 1) + 4 * (i >> 1);
                    w.x = Ty::pack(fmaf(s, sc_code_f(vw[0], sh), z), fmaf(s, sc_code_f(vw[1], sh), z));
                    w.y = Ty::pack(fmaf(s, sc_code_f(vw[2], sh), z), fmaf(s, sc_code_f(vw[3], sh), z));
                }
                *reinterpret_cast<uint2*>(ov + o) = w;
            }
        }
    }
}

}  // namespace sv
