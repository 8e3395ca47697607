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
// while the scale is a normal number).  Where it comes that close to a half
// (both sides have few bits, so that of 128 elements one often lies on it), the
// remainder decides: d - code * scale has no rounding error (a multiple of d's
// last bit and no larger than d), and a quotient that is not a half lies
// further from one than half its last bit, so that the exact quotient and the
// rounded one fall on the same side.
__device__ __forceinline__ void sc_near(float& c, float d, float scale, float half) {
    const float r = fmaf(-c, scale, d), a = fabsf(r);
    c += copysignf(a > half ? 0.75f : a == half ? 0.5f : 0.25f, r);
}
// ... and where the scale is too small for a reciprocal.
__device__ __noinline__ float sc_divided(float d, float scale) {
    const float x = scale > 0.f ? fminf(rintf(__fdiv_rn(d, scale)), 15.f) : 0.f;
    return x >= 0.f ? x : 0.f;
}
__device__ __forceinline__ void sc_codes4(uint64_t x01, uint64_t x23, float zero, float scale, float inv,
                                          uint64_t& c01, uint64_t& c23) {
    const uint64_t nz = f2_pack(-zero, -zero), i2 = f2_pack(inv, inv), minus = f2_pack(-1.f, -1.f);
    const uint64_t up = f2_pack(12582912.f, 12582912.f), down = f2_pack(-12582912.f, -12582912.f);
    const uint64_t d01 = f2_add(x01, nz), d23 = f2_add(x23, nz);
    const uint64_t q01 = f2_mul(d01, i2), q23 = f2_mul(d23, i2);
    c01 = f2_add(f2_add(q01, up), down);
    c23 = f2_add(f2_add(q23, up), down);
    float e0, e1, e2, e3;
    f2_unpack(f2_fma(c01, minus, q01), e0, e1);
    f2_unpack(f2_fma(c23, minus, q23), e2, e3);
    const float off = fmaxf(fmaxf(fabsf(e0), fabsf(e1)), fmaxf(fabsf(e2), fabsf(e3)));
    if (off >= 0.49998f || inv != inv) {
        float c[4], d[4];
        f2_unpack(c01, c[0], c[1]);
        f2_unpack(c23, c[2], c[3]);
        f2_unpack(d01, d[0], d[1]);
        f2_unpack(d23, d[2], d[3]);
        if (inv == inv) {
#pragma unroll
            for (int i = 0; i < 4; ++i) sc_near(c[i], d[i], scale, 0.5f * scale);
            c01 = f2_add(f2_add(f2_pack(c[0], c[1]), up), down);
            c23 = f2_add(f2_add(f2_pack(c[2], c[3]), up), down);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) c[i] = sc_divided(d[i], scale);
            c01 = f2_pack(c[0], c[1]);
            c23 = f2_pack(c[2], c[3]);
        }
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
    uint32_t have = 0xffu;
    {
        const typename Ty::T* kp = static_cast<const typename Ty::T*>(P.k) + static_cast<size_t>(h) * D + 4 * l;
        const typename Ty::T* vp = static_cast<const typename Ty::T*>(P.v) + static_cast<size_t>(h) * D + 4 * l;
        const size_t row = static_cast<size_t>(b) * P.n;
        if (!P.nodes && from <= g * 8 && g * 8 + 8 <= to) {  // a whole group of rows side by side
            const size_t o = (row + (p0 - len)) * static_cast<size_t>(P.stride);
            kp += o;
            vp += o;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                raw[i] = *reinterpret_cast<const uint2*>(kp);
                raw[8 + i] = *reinterpret_cast<const uint2*>(vp);
                kp += P.stride;
                vp += P.stride;
            }
        } else {
            have = 0;
            int node[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int t = g * 8 + i;
                node[i] = t >= from && t < to ? sc_node(P, b, t0 + t - len) : -1;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                raw[i] = raw[8 + i] = make_uint2(0u, 0u);
                if (node[i] >= 0 && node[i] < P.n) {
                    have |= 1u << i;
                    const size_t o = (row + node[i]) * static_cast<size_t>(P.stride);
                    raw[i] = *reinterpret_cast<const uint2*>(kp + o);
                    raw[8 + i] = *reinterpret_cast<const uint2*>(vp + o);
                }
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
    if (l < 16) {
        const int i = 8 * (l & 1) + 4 * ((l >> 1) & 1) + 2 * ((l >> 2) & 1) + ((l >> 3) & 1);  // the lane's row
        if ((have >> (i & 7)) & 1u)
            *reinterpret_cast<uint32_t*>((i < 8 ? blkp : vblk) + T * (D / 2) + (g * 8 + (i & 7)) * 4) = par;
    }
    uint32_t before = 0;
    uint64_t vacc[2][2];  // dims {0, 1} and {2, 3} of the lane: the even and the odd tokens' codes
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int src = ((i >> 3) & 1) | ((i >> 1) & 2) | ((i << 1) & 4) | ((i << 3) & 8);
        const uint32_t p = __shfl_sync(mask, par, src, LPI);
        const float iv = __shfl_sync(mask, inv, src, LPI);
        uint64_t c01, c23;
        sc_codes4(f2_pack(Ty::lo(raw[i].x), Ty::hi(raw[i].x)), f2_pack(Ty::lo(raw[i].y), Ty::hi(raw[i].y)), Ty::hi(p),
                  Ty::lo(p), iv, c01, c23);
        if (i < 8) {
            // a key row's word w: dims 8w.. from lanes 2w (low byte of each half) and 2w+1
            float lo, hi;
            f2_unpack(f2_fma(f2_pack(16.f, 16.f), c23, c01), lo, hi);
            uint32_t w = __byte_perm(sc_bits(lo), sc_bits(hi), (l & 1) ? 0x4707 : 0x7470) &
                         ((l & 1) ? 0xFF00FF00u : 0x00FF00FFu);
            w |= __shfl_xor_sync(mask, w, 1);
            if (i & 1) {  // the even lanes store the token before, the odd ones this
                const int t = i - 1 + (l & 1);
                if ((have >> t) & 1u)
                    *reinterpret_cast<uint32_t*>(blkp + (g * 8 + t) * (D / 2) + (l >> 1) * 4) = (l & 1) ? w : before;
            }
            before = w;
        } else {
            const int e = i & 1, m = (i & 7) >> 1;  // token 2m + e: bits 16e + 4m
            const float f = m == 1 ? 16.f : m == 2 ? 256.f : 4096.f;
            vacc[0][e] = m == 0 ? c01 : f2_fma(f2_pack(f, f), c01, vacc[0][e]);
            vacc[1][e] = m == 0 ? c23 : f2_fma(f2_pack(f, f), c23, vacc[1][e]);
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
    const int g = static_cast<int>(p0 - t0) >> 3;
    // the group's words and parameters; nothing where its block cannot be read
    uint32_t kw[8], vw[4], kp[8], vp[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) kw[i] = kp[i] = vp[i] = 0u;
#pragma unroll
    for (int q = 0; q < 4; ++q) vw[q] = 0u;
    if (blkp) {
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
            const uint4 a = *reinterpret_cast<const uint4*>(blkp + T * (D / 2) + (g * 8 + i) * 4);
            const uint4 e = *reinterpret_cast<const uint4*>(vblk + T * (D / 2) + (g * 8 + i) * 4);
            kp[i] = a.x, kp[i + 1] = a.y, kp[i + 2] = a.z, kp[i + 3] = a.w;
            vp[i] = e.x, vp[i + 1] = e.y, vp[i + 2] = e.z, vp[i + 3] = e.w;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            kw[i] = *reinterpret_cast<const uint32_t*>(blkp + (g * 8 + i) * (D / 2) + (l >> 1) * 4);
#pragma unroll
        for (int q = 0; q < 4; ++q)
            vw[q] = *reinterpret_cast<const uint32_t*>(vblk + (4 * l + q) * (T / 2) + g * 4);
    }
    // rows of the group that are read, and of them those that hold a token
    uint32_t rows = 0, in = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int t = g * 8 + i;
        const long long pos = t0 + t;
        if (t >= from && t < to) rows |= 1u << i;
        if (pos >= 0 && pos < len) in |= 1u << i;
    }
    typename Ty::T* ok = static_cast<typename Ty::T*>(P.out_k);
    typename Ty::T* ov = static_cast<typename Ty::T*>(P.out_v);
    const size_t step = static_cast<size_t>(c.kv_heads) * D;
    // (of the group's first row, which may lie before the range)
    const long long o0 = ((static_cast<long long>(b) * P.n + (p0 - first)) * c.kv_heads + h) * D + 4 * l;
    const uint64_t down = f2_pack(-8388608.f, -8388608.f);
    const uint32_t sel = 0x7540u + (l & 1);  // a byte of the codes below 2^23's upper bytes
    uint32_t vlo[4], vhi[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        vlo[q] = vw[q] & 0x0F0F0F0Fu;
        vhi[q] = (vw[q] >> 4) & 0x0F0F0F0Fu;
    }
    auto value = [&](uint32_t a, uint32_t e, uint64_t s2, uint64_t z2) {  // two codes as floats above 2^23
        float x, y;
        f2_unpack(f2_fma(s2, f2_add(f2_pack(__uint_as_float(a), __uint_as_float(e)), down), z2), x, y);
        return Ty::pack(x, y);
    };
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (!((rows >> i) & 1u)) continue;
        const bool token = (in >> i) & 1u;
        const size_t o = static_cast<size_t>(o0 + static_cast<long long>(i) * static_cast<long long>(step));
        const uint32_t fill = token && bad ? 0x7fff7fffu : 0u;
        if (ok) {
            const float s = Ty::lo(kp[i]), z = Ty::hi(kp[i]);
            const uint64_t s2 = f2_pack(s, s), z2 = f2_pack(z, z);
            const uint32_t lo = kw[i] & 0x0F0F0F0Fu, hi = (kw[i] >> 4) & 0x0F0F0F0Fu;
            uint2 y = make_uint2(value(__byte_perm(lo, 0x4B000000u, sel), __byte_perm(lo, 0x4B000000u, sel + 2), s2, z2),
                                 value(__byte_perm(hi, 0x4B000000u, sel), __byte_perm(hi, 0x4B000000u, sel + 2), s2, z2));
            if (!token || bad) y = make_uint2(fill, fill);
            *reinterpret_cast<uint2*>(ok + o) = y;
        }
        if (ov) {
            const float s = Ty::lo(vp[i]), z = Ty::hi(vp[i]);
            const uint64_t s2 = f2_pack(s, s), z2 = f2_pack(z, z);
            // token i: nibble (i / 2) of the half i % 2, so byte i / 4 + 2 (i % 2), its upper half for i / 2 odd
            const uint32_t vs = 0x7540u + (i >> 2) + 2 * (i & 1);
            uint32_t x[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) x[q] = __byte_perm(((i >> 1) & 1) ? vhi[q] : vlo[q], 0x4B000000u, vs);
            uint2 y = make_uint2(value(x[0], x[1], s2, z2), value(x[2], x[3], s2, z2));
            if (!token || bad) y = make_uint2(fill, fill);
            *reinterpret_cast<uint2*>(ov + o) = y;
        }
    }
}

}  // namespace sv
