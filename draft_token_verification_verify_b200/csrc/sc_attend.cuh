// Attention of the scored positions over the 4-bit cache and over themselves.
//
// For one sequence and key/value head the rows are the n positions x the
// group's query heads.  A cached key row stands for zero + scale * code, so
//   q . k = scale * (q . code) + zero * sum(q)
// and the codes go to the tensor cores as they are; a cached value row is
// folded into the softmax weight, p' = p * scale, with codes centred to
// code - 8 (exact) and sum p (zero + 8 scale) added at the end.
//
// K_attend<DT, D>: 16 rows a block (m16n8k16 MMAs), four warps a CTA, each
// warp on its own tiles of 64 tokens with its own ring of bulk copies, no
// barrier between the warps until their (max, sum, output) are merged at the
// end of a segment.  The fragment order is chosen so that a lane's operands
// are contiguous in the block: 16 (8) bytes of a key row hold the lane's share
// of the whole dot product, 8 bytes of a value row its 16 tokens.
//
// The work: a segment is (sequence, head, block of 16 rows) and has
// ceil(len / 64) tiles of the cache and ceil(n / 64) units of scored
// positions.  The segments' tiles in a row are cut into equal ranges, one for
// each CTA of a single wave; a segment that is cut leaves partial sums that
// K_join adds in the order of the parts.
#pragma once

#include "sc_common.cuh"

namespace sv {

constexpr int SC_WARPS = 4;
constexpr int SC_NT = SC_WARPS * 32;
constexpr int SC_ROWS = 16;   // rows of a block
constexpr int SC_STAGES = 2;  // tiles in flight for each warp
constexpr int SC_MIN_TILES = 4;  // tiles of a CTA's range at least

struct AttendParams {
    CacheView c;
    const void* q;
    const void* k_new;  // null: the cached context alone
    const void* v_new;
    const int32_t* parents;
    long long q_stride, kv_stride;  // elements between tokens
    int B, n, q_heads, group;
    int rows, row_blocks;  // n * group, in blocks of SC_ROWS (or the tensor-memory kernel's width)
    float scale;
    void* out;
    float* out_lse;
    // workspace
    float* part_o;   // [grid][2][rows of a block][D]
    float2* part_ml; // [grid][2][rows of a block]
    int4* desc;      // [grid]: {segment cut here that begins in this CTA: b, head * row_blocks + block, parts, error}
    unsigned long long timeout_ns;
    int test_hook;
    int32_t* out_status;
};

// Units of a sequence: its cache tiles and the units of its scored positions.
__device__ __forceinline__ int sc_len(const AttendParams& P, int b, bool* bad) {
    const int len = P.c.lens[b];
    *bad = len > sc_capacity(P.c);
    return (len < 0 || *bad) ? 0 : len;
}
template <int TILE>
__device__ __forceinline__ int sc_new_units(const AttendParams& P) {
    return P.k_new ? (P.n + TILE - 1) / TILE : 0;
}
template <int TILE>
__device__ __forceinline__ int sc_units(const AttendParams& P, int b) {
    bool bad;
    const int u = (sc_len(P, b, &bad) + TILE - 1) / TILE + sc_new_units<TILE>(P);
    return u > 0 ? u : 1;
}

// A CTA's range of the segments' units, found by all its threads.
struct Range {
    long long total, chunk, g0, g1;  // units in all; of a CTA; this CTA's
    int b;                           // sequence that holds g0
    long long before;                // units before that sequence
};

template <int NT, int TILE>
__device__ __forceinline__ Range sc_range(const AttendParams& P, int min_units) {
    __shared__ long long scan[NT / 32];
    __shared__ long long found[2];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (P.B + NT - 1) / NT;
    const long long segs = static_cast<long long>(P.c.kv_heads) * P.row_blocks;
    long long mine = 0;
    for (int b = tid * per; b < (tid + 1) * per && b < P.B; ++b) mine += sc_units<TILE>(P, b);
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    long long base = 0, total = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
        if (w < warp) base += scan[w];
        total += scan[w];
    }
    Range r;
    r.total = total * segs;
    r.chunk = (r.total + gridDim.x - 1) / gridDim.x;
    if (r.chunk < min_units) r.chunk = min_units;
    r.g0 = r.chunk * blockIdx.x;
    r.g1 = r.g0 + r.chunk < r.total ? r.g0 + r.chunk : r.total;
    long long at = (base + incl - mine) * segs;
    if (r.g0 < r.g1 && r.g0 >= at && r.g0 < at + mine * segs) {
        int b = tid * per;
        for (;; ++b) {
            const long long u = sc_units<TILE>(P, b) * segs;
            if (r.g0 < at + u) break;
            at += u;
        }
        found[0] = b;
        found[1] = at;
    }
    __syncthreads();
    r.b = static_cast<int>(found[0]);
    r.before = found[1];
    __syncthreads();
    return r;
}

// A walk over the parts of segments in a CTA's range.
template <int TILE>
struct Walk {
    int b, hr;       // sequence; head * row_blocks + row block
    int units, len;  // of the sequence
    int u0, u1;      // the range's share of the segment's units: [u0, u1)
    int left;        // units of the range behind this part
    int u;           // for the caller: the unit it is at
    bool bad;        // a length above the capacity

    __device__ __forceinline__ void sequence(const AttendParams& P) {
        units = sc_units<TILE>(P, b);
        len = sc_len(P, b, &bad);
    }
    __device__ __forceinline__ void begin(const AttendParams& P, const Range& r) {
        b = r.b;
        sequence(P);
        const long long in = r.g0 - r.before;
        hr = static_cast<int>(in / units);
        u0 = static_cast<int>(in - static_cast<long long>(hr) * units);
        left = static_cast<int>(r.g1 - r.g0);
        u1 = units - u0 < left ? units : u0 + left;
        left -= u1 - u0;
    }
    // The next segment; false behind the range.
    __device__ __forceinline__ bool next(const AttendParams& P) {
        if (left <= 0) return false;
        if (++hr == P.c.kv_heads * P.row_blocks) {
            hr = 0;
            ++b;
            sequence(P);
        }
        u0 = 0;
        u1 = units < left ? units : left;
        left -= u1;
        return true;
    }
    // Whether this part is the whole segment.
    __device__ __forceinline__ bool whole() const { return u0 == 0 && u1 == units; }
    // CTAs that hold parts of a segment begun here and cut by the range's end.
    __device__ __forceinline__ int parts(int chunk) const { return 1 + (units - u1 + chunk - 1) / chunk; }
};

// Row `r` of segment (b, head): its element offset in [B][n][q_heads].
__device__ __forceinline__ size_t sc_out_row(const AttendParams& P, int b, int head, int r) {
    const int node = r / P.group, g = r - node * P.group;
    return (static_cast<size_t>(b) * P.n + node) * P.q_heads + head * P.group + g;
}

template <int D>
struct AttendSmem {
    // Blocks of a tile lie `stride` bytes apart: shorter blocks are padded so
    // that the four quarter-tiles of a value read fall into different banks.
    static constexpr int TILE = 2 * sc_half_bytes<D>(SC_BLOCK) + 128;
    static constexpr int RING = SC_WARPS * SC_STAGES * TILE;
    static constexpr int MERGE_ROW = D + 4;  // floats
    static constexpr int MERGE = SC_ROWS * MERGE_ROW * 4;  // a warp's output, or its staged value rows
    static constexpr int ML = SC_WARPS * SC_ROWS * 8;
    static constexpr int BYTES = RING + SC_WARPS * MERGE + ML + SC_WARPS * SC_STAGES * 8 + 64;
    static_assert(SC_ROWS * (D + 8) * 2 <= MERGE, "staged value rows fit the merge buffer");
};

template <int DT, int D>
__global__ void __launch_bounds__(SC_NT, 2) sc_attend_kernel(const __grid_constant__ AttendParams P) {
    using Ty = SC<DT>;
    using Sm = AttendSmem<D>;
    using T = typename Ty::T;
    constexpr int KS = D / 16;   // k-steps of a dot product
    constexpr int KW = D / 32;   // 32-bit words of a lane's share of a key row
    constexpr int NV = D / 8;    // n-tiles of the output
    extern __shared__ __align__(128) unsigned char sc_raw[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int r8 = lane >> 2, q4 = lane & 3;
    unsigned char* ring = sc_raw + warp * SC_STAGES * Sm::TILE;
    float* merge = reinterpret_cast<float*>(sc_raw + Sm::RING + warp * Sm::MERGE);
    float2* ml = reinterpret_cast<float2*>(sc_raw + Sm::RING + SC_WARPS * Sm::MERGE);
    uint64_t* bars = reinterpret_cast<uint64_t*>(sc_raw + Sm::RING + SC_WARPS * Sm::MERGE + Sm::ML) +
                     warp * SC_STAGES;
    const CacheView& c = P.c;

    pdl_launch_dependents();
    const Range R = sc_range<SC_NT, SC_BLOCK>(P, SC_MIN_TILES);
    int error = 0;
    if (tid == 0) P.desc[blockIdx.x] = make_int4(-1, 0, 0, 0);
    if (R.g0 >= R.g1) return;
    if (lane == 0) {
        for (int s = 0; s < SC_STAGES; ++s) mbar_init(&bars[s], 1);
        fence_mbar_init();
    }
    __syncwarp();

    const int nb = SC_BLOCK >> c.log2_block;  // blocks of a tile
    const int bstride = 2 * sc_half_bytes<D>(c.block) + (nb == 1 ? 0 : nb == 2 ? 64 : 32);
    const float sl = P.scale * SC_LOG2E;

    // ---- the copies: tile `iw` of this warp is issued SC_STAGES tiles ahead ----
    Walk<SC_BLOCK> iw;
    iw.begin(P, R);
    iw.u = iw.u0 + warp;
    bool more = true;
    int ahead_id = 0, ahead_sub = 0;
    uint32_t bad_stage = 0;  // bit s: a page of stage s was out of range
    auto settle = [&]() {    // to the next cache tile at or behind iw.u
        while (more) {
            if (iw.u < iw.u1 && iw.u * SC_BLOCK < iw.len) break;
            more = iw.next(P);
            iw.u = iw.u0 + warp;
        }
        if (more && lane < nb) {  // lane j fetches block j of the tile
            const int t = iw.u * SC_BLOCK + (lane << c.log2_block);
            ahead_id = t < iw.len ? __ldg(c.table + static_cast<size_t>(iw.b) * c.max_pages + (t >> c.log2_page)) : -2;
            ahead_sub = (t & (c.page_size - 1)) >> c.log2_block;
        }
    };
    settle();
    int issued = 0, used = 0;
    auto issue = [&]() {
        if (!more) return;
        const int s = issued % SC_STAGES;
        const int head = iw.hr / P.row_blocks;
        const uint32_t bytes = 2 * sc_half_bytes<D>(c.block);
        const bool mine = lane < nb && ahead_id != -2;
        const bool ok = mine && ahead_id >= 0 && ahead_id < c.num_pages && !P.test_hook;
        const unsigned got = __ballot_sync(0xffffffffu, ok);
        const unsigned want = __ballot_sync(0xffffffffu, mine);
        bad_stage = (bad_stage & ~(1u << s)) | ((got != want && !P.test_hook) ? 1u << s : 0u);
        if (lane == 0) mbar_arrive_expect_tx(&bars[s], P.test_hook ? bytes : bytes * __popc(got));
        __syncwarp();
        if (ok) bulk_g2s(ring + s * Sm::TILE + lane * bstride, sc_block_ptr<D>(c, ahead_id, head, ahead_sub), bytes, &bars[s]);
        ++issued;
        iw.u += SC_WARPS;
        settle();
    };
    for (int s = 0; s < SC_STAGES; ++s) issue();

    Walk<SC_BLOCK> w;
    w.begin(P, R);
    for (bool go = true; go; go = w.next(P)) {
        const int head = w.hr / P.row_blocks, row0 = (w.hr % P.row_blocks) * SC_ROWS;
        // ---- this segment's queries, in fragment order ----
        uint32_t qa[KS][4];
        float qs[2] = {0.f, 0.f};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int row = row0 + r8 + 8 * e;
            const bool in = row < P.rows;
            const int node = row / P.group, g = row - node * P.group;
            const T* src = static_cast<const T*>(P.q) +
                           (static_cast<long long>(w.b) * P.n + node) * P.q_stride +
                           static_cast<long long>(head * P.group + g) * D + q4 * (D / 4);
#pragma unroll
            for (int i = 0; i < KS / 2; ++i) {
                const uint4 x = in ? *reinterpret_cast<const uint4*>(src + 8 * i) : make_uint4(0u, 0u, 0u, 0u);
                qa[2 * i][e] = x.x;
                qa[2 * i][2 + e] = x.y;
                qa[2 * i + 1][e] = x.z;
                qa[2 * i + 1][2 + e] = x.w;
                qs[e] += (Ty::lo(x.x) + Ty::hi(x.x)) + (Ty::lo(x.y) + Ty::hi(x.y)) + (Ty::lo(x.z) + Ty::hi(x.z)) +
                         (Ty::lo(x.w) + Ty::hi(x.w));
            }
            qs[e] += __shfl_xor_sync(0xffffffffu, qs[e], 1);
            qs[e] += __shfl_xor_sync(0xffffffffu, qs[e], 2);
        }
        float o[NV][4];
#pragma unroll
        for (int u = 0; u < NV; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[u][i] = 0.f;
        float m[2] = {SC_NEG_INF, SC_NEG_INF}, l[2] = {0.f, 0.f}, z[2] = {0.f, 0.f};
        if (w.bad) l[0] = l[1] = __int_as_float(0x7fffffff);  // a length above the capacity

        // A new maximum rescales what was summed, but only where it passes the
        // reference by 2^8: until then the weights just exceed 1.
        auto reference = [&](float mx, int e) {
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            const bool up = mx > m[e] + 8.f;  // also from -inf
            if (__any_sync(0xffffffffu, up)) {
                const float f = up ? ex2(m[e] - mx) : 1.f;
                if (up) m[e] = mx;
                l[e] *= f;
                z[e] *= f;
#pragma unroll
                for (int u = 0; u < NV; ++u) {
                    o[u][2 * e] *= f;
                    o[u][2 * e + 1] *= f;
                }
            }
            return m[e] == SC_NEG_INF ? 0.f : m[e];
        };

        const int first = w.u0 + warp;
        for (int u = first; u < w.u1; u += SC_WARPS) {
            if (u * SC_BLOCK < w.len) {
                // ---- a tile of 64 cached tokens ----
                const int s = used % SC_STAGES;
                if (!error) {
                    const bool got = mbar_wait_bounded(&bars[s], (used / SC_STAGES) & 1, P.timeout_ns);
                    error = !__all_sync(0xffffffffu, got);
                }
                if (error || ((bad_stage >> s) & 1u)) l[0] = l[1] = __int_as_float(0x7fffffff);
                if (error) continue;  // nothing more is waited for
                ++used;
                const int valid = w.len - u * SC_BLOCK < SC_BLOCK ? w.len - u * SC_BLOCK : SC_BLOCK;
                const unsigned char* tile = ring + s * Sm::TILE;
                const int Tb = c.block;
                float x[8][4];
                {
                    // scores: lane r8 of n-tile t takes token 16 (r8 / 2) + 2 t + r8 % 2, so that
                    // the accumulators of a lane are the 16 tokens 16 q4 .. 16 q4 + 15
                    const int tk = 16 * (r8 >> 1);
                    const unsigned char* krow = tile + (tk >> c.log2_block) * bstride +
                                                ((tk & (Tb - 1)) + (r8 & 1)) * (D / 2) + q4 * (D / 8);
#pragma unroll
                    for (int t4 = 0; t4 < 8; t4 += 4) {
                        uint32_t kw[4][KW];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const unsigned char* a = krow + (t4 + i) * D;
                            if constexpr (KW == 4) {
                                const uint4 v = *reinterpret_cast<const uint4*>(a);
                                kw[i][0] = v.x, kw[i][1] = v.y, kw[i][2] = v.z, kw[i][3] = v.w;
                            } else {
                                const uint2 v = *reinterpret_cast<const uint2*>(a);
                                kw[i][0] = v.x, kw[i][1] = v.y;
                            }
#pragma unroll
                            for (int j = 0; j < 4; ++j) x[t4 + i][j] = 0.f;
                        }
#pragma unroll
                        for (int k = 0; k < KS; ++k)
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const uint32_t wd = kw[i][k >> 1];
                                if constexpr (DT == 0)
                                    sc_mma<0>(x[t4 + i], qa[k], sc_codes_bf16(wd, 2 * (k & 1)),
                                              sc_codes_bf16(wd, 2 * (k & 1) + 1));
                                else
                                    sc_mma<1>(x[t4 + i], qa[k], sc_center_f16(sc_codes_f16(wd, 2 * (k & 1))),
                                              sc_center_f16(sc_codes_f16(wd, 2 * (k & 1) + 1)));
                            }
                    }
                    const int tq = 16 * q4;
                    const unsigned char* kblk = tile + (tq >> c.log2_block) * bstride;
                    const unsigned char* par = kblk + Tb * (D / 2) + (tq & (Tb - 1)) * 4;
                    float mx[2] = {SC_NEG_INF, SC_NEG_INF};
#pragma unroll
                    for (int t = 0; t < 8; t += 2) {
                        const uint4 pr = *reinterpret_cast<const uint4*>(par + t * 8);
                        const uint32_t pw[4] = {pr.x, pr.y, pr.z, pr.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float s1 = Ty::lo(pw[i]);
                            const float f = s1 * sl;
                            // codes enter as 128 + code (bf16) or code - 8 (fp16)
                            const float zz = fmaf(DT == 0 ? -128.f : 8.f, s1, Ty::hi(pw[i])) * sl;
                            float* a = x[t + (i >> 1)];
                            a[i & 1] = fmaf(f, a[i & 1], zz * qs[0]);
                            a[2 + (i & 1)] = fmaf(f, a[2 + (i & 1)], zz * qs[1]);
                        }
                    }
                    if (valid < SC_BLOCK) {
#pragma unroll
                        for (int t = 0; t < 8; ++t)
#pragma unroll
                            for (int i = 0; i < 2; ++i)
                                if (tq + 2 * t + i >= valid) x[t][i] = x[t][2 + i] = SC_NEG_INF;
                    }
#pragma unroll
                    for (int t = 0; t < 8; ++t) {
                        mx[0] = fmaxf(mx[0], fmaxf(x[t][0], x[t][1]));
                        mx[1] = fmaxf(mx[1], fmaxf(x[t][2], x[t][3]));
                    }
                    const float m0 = reference(mx[0], 0), m1 = reference(mx[1], 1);
                    // softmax weights times the values' scales
                    const unsigned char* vblk = kblk + sc_half_bytes<D>(Tb);
                    const unsigned char* vpar = vblk + Tb * (D / 2) + (tq & (Tb - 1)) * 4;
                    uint32_t pa[4][4];
#pragma unroll
                    for (int t = 0; t < 8; t += 2) {
                        const uint4 pr = *reinterpret_cast<const uint4*>(vpar + t * 8);
                        const uint32_t pw[4] = {pr.x, pr.y, pr.z, pr.w};
#pragma unroll
                        for (int h2 = 0; h2 < 2; ++h2) {
                            float ps[2][2];
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const uint32_t pp = pw[2 * h2 + i];
                                float s1 = Ty::lo(pp), z1 = fmaf(8.f, s1, Ty::hi(pp));
                                if (valid < SC_BLOCK && tq + 2 * (t + h2) + i >= valid) s1 = z1 = 0.f;
                                const float p0 = ex2(x[t + h2][i] - m0), p1 = ex2(x[t + h2][2 + i] - m1);
                                l[0] += p0;
                                l[1] += p1;
                                z[0] = fmaf(p0, z1, z[0]);
                                z[1] = fmaf(p1, z1, z[1]);
                                ps[0][i] = p0 * s1;
                                ps[1][i] = p1 * s1;
                            }
                            // rounded to bf16 whatever the cache's type: p * scale keeps fp32's range there
                            pa[t >> 1][2 * h2] = SC<0>::pack(ps[0][0], ps[0][1]);
                            pa[t >> 1][2 * h2 + 1] = SC<0>::pack(ps[1][0], ps[1][1]);
                        }
                    }
                    const unsigned char* vrow = vblk + r8 * (Tb / 2) + (tq & (Tb - 1)) / 2;
#pragma unroll
                    for (int u4 = 0; u4 < NV; u4 += 4) {
                        uint2 vw[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            vw[i] = *reinterpret_cast<const uint2*>(vrow + (u4 + i) * 8 * (Tb / 2));
#pragma unroll
                        for (int k = 0; k < 4; ++k)
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const uint32_t wd = k < 2 ? vw[i].x : vw[i].y;
                                sc_mma<0>(o[u4 + i], pa[k], sc_center_bf16(sc_codes_bf16(wd, 2 * (k & 1))),
                                          sc_center_bf16(sc_codes_bf16(wd, 2 * (k & 1) + 1)));
                            }
                    }
                }
                __syncwarp();
                issue();  // into the stage just read
            } else if (P.k_new) {
                // ---- up to 64 of the scored positions, 16 at a time ----
                const int ub = (u - (w.len + SC_BLOCK - 1) / SC_BLOCK) * SC_BLOCK;
                const int32_t* par = P.parents ? P.parents + static_cast<size_t>(w.b) * (P.n - 1) : nullptr;
                if (par) {
                    int bad = 0;
                    for (int i = 1 + lane; i < P.n; i += 32) bad |= par[i - 1] < 0 || par[i - 1] >= i;
                    if (__any_sync(0xffffffffu, bad)) {  // no such tree
                        l[0] = l[1] = __int_as_float(0x7fffffff);
                        continue;
                    }
                }
                for (int j0 = ub; j0 < ub + SC_BLOCK && j0 < P.n; j0 += 16) {
                    float x[2][4];
                    const long long tok = static_cast<long long>(w.b) * P.n;
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const int j = j0 + 8 * t + r8;
                        const bool in = j < P.n;
                        const T* src = static_cast<const T*>(P.k_new) + (tok + j) * P.kv_stride +
                                       static_cast<long long>(head) * D + q4 * (D / 4);
#pragma unroll
                        for (int i = 0; i < 4; ++i) x[t][i] = 0.f;
#pragma unroll
                        for (int i = 0; i < KS / 2; ++i) {
                            const uint4 kx = in ? *reinterpret_cast<const uint4*>(src + 8 * i) : make_uint4(0u, 0u, 0u, 0u);
                            sc_mma<DT>(x[t], qa[2 * i], kx.x, kx.y);
                            sc_mma<DT>(x[t], qa[2 * i + 1], kx.z, kx.w);
                        }
                    }
                    // value rows of the 16 positions, zeros behind the last; a row that is not
                    // finite is left out of the MMAs, where it would reach the rows that do not
                    // see it, and added by itself
                    T* vs = reinterpret_cast<T*>(merge);
                    uint32_t odd = 0;
                    __syncwarp();
                    for (int i = lane; i < 16 * (D / 8); i += 32) {
                        const int jr = i / (D / 8), dc = i % (D / 8);
                        uint4 vx = make_uint4(0u, 0u, 0u, 0u);
                        if (j0 + jr < P.n)
                            vx = *reinterpret_cast<const uint4*>(static_cast<const T*>(P.v_new) +
                                                                 (tok + j0 + jr) * P.kv_stride +
                                                                 static_cast<long long>(head) * D + dc * 8);
                        const uint32_t vv[4] = {vx.x, vx.y, vx.z, vx.w};
                        bool fine = true;
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            fine &= fabsf(Ty::lo(vv[k])) < __builtin_huge_valf() && fabsf(Ty::hi(vv[k])) < __builtin_huge_valf();
                        if (!fine) odd |= 1u << jr;
                        *reinterpret_cast<uint4*>(vs + jr * (D + 8) + dc * 8) = vx;
                    }
                    odd = __reduce_or_sync(0xffffffffu, odd);
                    if (odd) {
                        for (int i = lane; i < 16 * (D / 8); i += 32)
                            if ((odd >> (i / (D / 8))) & 1u)
                                *reinterpret_cast<uint4*>(vs + (i / (D / 8)) * (D + 8) + (i % (D / 8)) * 8) =
                                    make_uint4(0u, 0u, 0u, 0u);
                    }
                    __syncwarp();
                    float mx[2] = {SC_NEG_INF, SC_NEG_INF};
                    uint32_t seen = 0;  // bit 4 e + 2 t + i: row e sees position 8 t + 2 q4 + i
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int row = row0 + r8 + 8 * e;
                        const int node = row / P.group;
#pragma unroll
                        for (int t = 0; t < 2; ++t)
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const int j = j0 + 8 * t + 2 * q4 + i;
                                bool see = row < P.rows && j < P.n && j <= node;
                                if (see && par) {  // climb from the node to the position, or past it
                                    int a = node;
                                    while (a > j) a = par[a - 1];
                                    see = a == j;
                                }
                                seen |= see ? 1u << (4 * e + 2 * t + i) : 0u;
                                x[t][2 * e + i] = see ? x[t][2 * e + i] * sl : SC_NEG_INF;
                                mx[e] = fmaxf(mx[e], x[t][2 * e + i]);
                            }
                    }
                    const float mm[2] = {reference(mx[0], 0), reference(mx[1], 1)};
                    float p[2][4];
#pragma unroll
                    for (int t = 0; t < 2; ++t)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int e = i >> 1;
                            p[t][i] = (seen >> (4 * e + 2 * t + (i & 1))) & 1u ? ex2(x[t][i] - mm[e]) : 0.f;
                            l[e] += p[t][i];
                        }
                    const uint32_t pa[4] = {Ty::pack(p[0][0], p[0][1]), Ty::pack(p[0][2], p[0][3]),
                                            Ty::pack(p[1][0], p[1][1]), Ty::pack(p[1][2], p[1][3])};
#pragma unroll
                    for (int v = 0; v < NV; v += 2) {
                        uint32_t b4[4];
                        asm volatile(
                            "ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                            : "=r"(b4[0]), "=r"(b4[1]), "=r"(b4[2]), "=r"(b4[3])
                            : "r"(smem_u32(vs + (lane & 15) * (D + 8) + (v + (lane >> 4)) * 8)));
                        sc_mma<DT>(o[v], pa, b4[0], b4[1]);
                        sc_mma<DT>(o[v + 1], pa, b4[2], b4[3]);
                    }
                    for (; odd; odd &= odd - 1) {
                        const int jr = __ffs(odd) - 1;
                        const T* src = static_cast<const T*>(P.v_new) + (tok + j0 + jr) * P.kv_stride +
                                       static_cast<long long>(head) * D;
                        const int from = (lane & ~3) | ((jr & 7) >> 1);  // the lane that holds the position's weights
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int bit = 4 * e + 2 * (jr >> 3) + (jr & 1);
                            const float mine = (jr >> 3) ? ((jr & 1) ? p[1][2 * e + 1] : p[1][2 * e])
                                                         : ((jr & 1) ? p[0][2 * e + 1] : p[0][2 * e]);
                            const float pe = __shfl_sync(0xffffffffu, mine, from);
                            const bool see = (__shfl_sync(0xffffffffu, seen, from) >> bit) & 1u;
#pragma unroll
                            for (int u8 = 0; u8 < NV; ++u8) {
                                const uint32_t vv = *reinterpret_cast<const uint32_t*>(src + u8 * 8 + 2 * q4);
                                if (see) {
                                    o[u8][2 * e] = fmaf(pe, Ty::lo(vv), o[u8][2 * e]);
                                    o[u8][2 * e + 1] = fmaf(pe, Ty::hi(vv), o[u8][2 * e + 1]);
                                }
                            }
                        }
                    }
                    __syncwarp();
                }
            }
        }

        // ---- merge the warps: 16 rows of (max, sum, output) ----
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
            l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
            z[e] += __shfl_xor_sync(0xffffffffu, z[e], 1);
            z[e] += __shfl_xor_sync(0xffffffffu, z[e], 2);
            const int r = r8 + 8 * e;
            if (q4 == 0) ml[warp * SC_ROWS + r] = make_float2(m[e], l[e]);
#pragma unroll
            for (int u = 0; u < NV; ++u)
                *reinterpret_cast<float2*>(merge + r * Sm::MERGE_ROW + u * 8 + 2 * q4) =
                    make_float2(o[u][2 * e] + z[e], o[u][2 * e + 1] + z[e]);
        }
        __syncthreads();
        const bool whole = w.whole();
        const int slot = blockIdx.x * 2 + (w.u0 == 0 ? 1 : 0);
        const float* all = reinterpret_cast<const float*>(sc_raw + Sm::RING);
        constexpr int PER = SC_NT / SC_ROWS;  // threads of a row
        const int r = tid / PER, cpart = tid % PER;
        float M = SC_NEG_INF, L = 0.f, wt[SC_WARPS];
#pragma unroll
        for (int i = 0; i < SC_WARPS; ++i) M = fmaxf(M, ml[i * SC_ROWS + r].x);
#pragma unroll
        for (int i = 0; i < SC_WARPS; ++i) {
            const float2 v = ml[i * SC_ROWS + r];
            wt[i] = v.x == SC_NEG_INF ? 0.f : ex2(v.x - M);
            L += v.x == SC_NEG_INF ? v.y : v.y * wt[i];  // (without a maximum the sum is 0 or NaN)
        }
        const int row = row0 + r;
        const float norm = whole ? (L == 0.f ? 0.f : 1.f / L) : 1.f;
        if (row < P.rows || !whole) {
            const size_t orow = whole ? sc_out_row(P, w.b, head, row) : 0;
#pragma unroll
            for (int i = 0; i < D / (4 * PER); ++i) {
                const int d = (i * PER + cpart) * 4;
                float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int k = 0; k < SC_WARPS; ++k) {
                    const float4 v = *reinterpret_cast<const float4*>(all + k * (Sm::MERGE / 4) + r * Sm::MERGE_ROW + d);
                    a.x = fmaf(wt[k], v.x, a.x);
                    a.y = fmaf(wt[k], v.y, a.y);
                    a.z = fmaf(wt[k], v.z, a.z);
                    a.w = fmaf(wt[k], v.w, a.w);
                }
                if (whole) {
                    uint2 y;
                    y.x = Ty::pack(a.x * norm, a.y * norm);
                    y.y = Ty::pack(a.z * norm, a.w * norm);
                    if (L != L) y = make_uint2(0x7fff7fffu, 0x7fff7fffu);
                    *reinterpret_cast<uint2*>(static_cast<T*>(P.out) + orow * D + d) = y;
                } else {
                    *reinterpret_cast<float4*>(P.part_o + (static_cast<size_t>(slot) * SC_ROWS + r) * D + d) = a;
                }
            }
            if (cpart == 0) {
                if (!whole)
                    P.part_ml[static_cast<size_t>(slot) * SC_ROWS + r] = make_float2(M, L);
                else if (P.out_lse)
                    P.out_lse[orow] = L == 0.f ? SC_NEG_INF : (M + log2f(L)) * SC_LN2;
            }
        }
        if (tid == 0 && w.u0 == 0 && !whole) {
            P.desc[blockIdx.x] = make_int4(w.b, w.hr, w.parts(static_cast<int>(R.chunk)), 0);
        }
        __syncthreads();  // the merge buffers are free
    }
    // no copy may land after the CTA is gone (after an error some are still under way)
    while (used < issued) {
        if (!mbar_wait_bounded(&bars[used % SC_STAGES], (used / SC_STAGES) & 1, P.timeout_ns)) error = 1;
        ++used;
    }
    if (error && lane == 0) P.desc[blockIdx.x].w = 1;
}

// K_join: block (i, j) adds the parts of the segment that is cut in CTA i and
// begins there, rows j, j + gridDim.y, ..., in the order of the parts.
constexpr int SC_JOIN_NT = 128;

template <int DT, int D>
__global__ void __launch_bounds__(SC_JOIN_NT) sc_join_kernel(const __grid_constant__ AttendParams P, int grid,
                                                            int block_rows) {
    using Ty = SC<DT>;
    pdl_wait_primary();
    if (blockIdx.x == 0 && blockIdx.y == 0 && P.out_status) {
        int err = 0;
        for (int i = threadIdx.x; i < grid; i += SC_JOIN_NT) err |= P.desc[i].w;
        err = __syncthreads_or(err);
        if (threadIdx.x == 0) *P.out_status = err ? -4 : 0;
    }
    const int4 d = P.desc[blockIdx.x];
    if (d.x < 0 || d.z == 0) return;
    const int head = d.y / P.row_blocks, row0 = (d.y % P.row_blocks) * block_rows;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    constexpr int V = D / 32;  // outputs of a lane
    for (int r = blockIdx.y * (SC_JOIN_NT / 32) + warp; r < block_rows && row0 + r < P.rows;
         r += gridDim.y * (SC_JOIN_NT / 32)) {
        float M = SC_NEG_INF;
        for (int p = lane; p < d.z; p += 32) {
            const int slot = (blockIdx.x + p) * 2 + (p == 0 ? 1 : 0);
            M = fmaxf(M, P.part_ml[static_cast<size_t>(slot) * block_rows + r].x);
        }
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, s));
        float L = 0.f, a[V];
#pragma unroll
        for (int i = 0; i < V; ++i) a[i] = 0.f;
#pragma unroll 4
        for (int p = 0; p < d.z; ++p) {
            const int slot = (blockIdx.x + p) * 2 + (p == 0 ? 1 : 0);
            const size_t at = static_cast<size_t>(slot) * block_rows + r;
            const float2 v = P.part_ml[at];
            const float wt = v.x == SC_NEG_INF ? 0.f : ex2(v.x - M);
            L += v.x == SC_NEG_INF ? v.y : v.y * wt;  // (without a maximum the sum is 0 or NaN)
            const float* src = P.part_o + at * D + lane * V;
#pragma unroll
            for (int i = 0; i < V; ++i) a[i] = fmaf(wt, src[i], a[i]);
        }
        const float norm = L == 0.f ? 0.f : 1.f / L;
        const size_t orow = sc_out_row(P, d.x, head, row0 + r);
        uint32_t y[V / 2];
#pragma unroll
        for (int i = 0; i < V / 2; ++i)
            y[i] = L != L ? 0x7fff7fffu : Ty::pack(a[2 * i] * norm, a[2 * i + 1] * norm);
#pragma unroll
        for (int i = 0; i < V / 2; ++i)
            reinterpret_cast<uint32_t*>(static_cast<typename Ty::T*>(P.out) + orow * D + lane * V)[i] = y[i];
        if (lane == 0 && P.out_lse) P.out_lse[orow] = L == 0.f ? SC_NEG_INF : (M + log2f(L)) * SC_LN2;
    }
}

}  // namespace sv
