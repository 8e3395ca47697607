// The attention on the 5th-generation tensor cores, transposed so that the
// few rows are the narrow side: with 128 cached tokens a tile,
//   S^T[token][row] = K codes [token][dim] . Q^T         (A: tensor memory)
//   O^T[dim][row]  += V codes [dim][token] . P^T         (A: tensor memory)
// Both A operands are 4-bit codes expanded by the CUDA cores straight into
// tensor memory, so the expanded tile never touches shared memory; the B
// operands (queries, softmax weights) are N = 16..80 rows wide.
//
// A code in the low byte of a 16-bit float is its value times the smallest
// subnormal (2^-133 in bf16, 2^-24 in fp16), exactly, and the tensor cores
// take subnormals: a mask is the whole expansion.  In bf16 the second code of
// a byte may stay four bits up (the exponent's lowest bit continues the
// mantissa there), as 16 times its value; its queries, or its token's weight,
// are divided by 16 instead.  Powers of two put the products back into range:
// queries are scaled by 2^64, weights by 2^64, S and O by 2^69 in fp32.
// (fp16 activations: queries stay as they are, and value codes are bf16
// numbers code - 8 under weights p * scale split into two bf16.)
//
// A token's scale and zero and a row's sum of q enter S after the product;
// p * scale weighs the value codes, and sum p * (zero + 8 scale) less 8 of the
// rounded weights is added at the end, all in fp32.  The reference maximum of a row is not moved until a score passes
// it by 2^8, so almost no tile touches the accumulated output.
//
// Roles of a CTA (one per SM): warp 16 bulk-copies the tiles' blocks, 17 issues
// the MMAs, 0-3 expand K, 4-7 expand V, 8-11 and 12-15 take the softmax (a
// thread is a token, its rows are registers): up to 32 rows the two groups
// take turns at the tiles, each with an output accumulator of its own; beyond,
// each takes half of the rows of every tile.  Every hand-over is an mbarrier
// with a bounded wait.
#pragma once

#include "sc_attend.cuh"

namespace sv {

constexpr int TC_TILE = 128;
constexpr int TC_NT = 20 * 32;  // the last two warps idle: registers move by groups of four warps
constexpr int TC_STAGES = 4;
constexpr int TC_MIN_TILES = 1;
constexpr int TC_MASK_WORDS = 12;  // 257 positions in tiles of 128

// ---- tensor memory and MMA wrappers -------------------------------------------

__device__ __forceinline__ void tc_alloc(uint32_t* slot, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(ncols)
                 : "memory");
}
__device__ __forceinline__ void tc_relinquish() {
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tc_dealloc(uint32_t addr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(ncols) : "memory");
}
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}
// D (tensor memory, fp32) = A (tensor memory) . B (shared memory) (+ D)
__device__ __forceinline__ void tc_mma(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
// 16 lanes x 32 columns: a thread writes columns 8 j + 2 (lane % 4) + {0, 1}
// of the lanes lane / 4 (x[4j], x[4j+1]) and lane / 4 + 8 (x[4j+2], x[4j+3]).
// (Four narrow stores: one of 16 registers in a row costs the expansion a move
// for each of them.)
__device__ __forceinline__ void tc_st16(uint32_t addr, const uint32_t (&x)[16]) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
        asm volatile("tcgen05.st.sync.aligned.16x256b.x1.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr + 8 * j),
                     "r"(x[4 * j]), "r"(x[4 * j + 1]), "r"(x[4 * j + 2]), "r"(x[4 * j + 3])
                     : "memory");
}
// 8 columns of the warp's 32 lanes, one lane a thread.
__device__ __forceinline__ void tc_ld8(uint32_t addr, float (&x)[8]) {
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(addr)
                 : "memory");
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tc_st8(uint32_t addr, const float (&x)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(addr),
                 "r"(__float_as_uint(x[0])), "r"(__float_as_uint(x[1])), "r"(__float_as_uint(x[2])),
                 "r"(__float_as_uint(x[3])), "r"(__float_as_uint(x[4])), "r"(__float_as_uint(x[5])),
                 "r"(__float_as_uint(x[6])), "r"(__float_as_uint(x[7]))
                 : "memory");
}
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void named_sync(int id, int threads) {
    asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ bool named_or(int id, int threads, bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %3, 0;\n\t"
        "barrier.cta.red.or.pred q, %1, %2, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(id), "r"(threads), "r"(static_cast<uint32_t>(x))
        : "memory");
    return __any_sync(0xffffffffu, r);
}
__device__ __forceinline__ float warp_max_f32(float x) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ bool tc_test(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return __all_sync(0xffffffffu, ok);
}
// Registers of a group of four warps.  The CTA starts with 640 x 96 = 61,440;
// 128 x (56 + 72 + 72 + 2 x 136) = 60,416 are given out.
template <int R>
__device__ __forceinline__ void regs_down() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void regs_up() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}

// Instruction descriptor: fp32 accumulator, A and B bf16 (1) or fp16 (0), both
// K-major, N = n, M = 128.
__host__ __device__ constexpr uint32_t tc_idesc(int bf16, int n) {
    return (1u << 4) | (static_cast<uint32_t>(bf16) << 7) | (static_cast<uint32_t>(bf16) << 10) |
           (static_cast<uint32_t>(n >> 3) << 17) | (8u << 24);
}
// K-major operand in shared memory, 128-byte swizzle, 8-row atoms of 1,024 bytes.
__device__ __forceinline__ uint64_t tc_desc(uint32_t saddr) {
    return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(1) << 16) |
           (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) |
           (static_cast<uint64_t>(2) << 61);
}

// N rows a block; ALT: the two softmax groups take turns at the tiles.
template <int DT, int D, int N_, bool ALT_>
struct TcShape {
    static constexpr int N = N_;
    static constexpr bool ALT = ALT_;
    static constexpr int NC = ALT ? N : N / 2;             // rows of a softmax thread
    static constexpr int ACC = ALT ? 2 : 1;                // output accumulators
    static constexpr int SR = N <= 48 ? 4 : 2;             // score buffers: tiles the MMAs may run ahead
    static constexpr int GROUP_WARPS = ALT ? 4 : 8;        // softmax warps of a tile
    static constexpr int STAGE = TC_TILE * (D + 8) + 256;  // blocks of 16 or 32 tokens are padded apart
    static constexpr int HALF = N * 128;                   // 64 elements of K for N rows
    static constexpr int Q = (D / 64) * HALF;              // one segment's queries
    static constexpr int PSPLIT = DT == 1 ? 2 : 1;         // fp16: the weights as a sum of two bf16
    static constexpr int PB = PSPLIT * 2 * HALF;           // one tile's weights
    static constexpr int OFF_P = 2 * Q;                    // (1,024-byte aligned regions first)
    static constexpr int OFF_RAW = OFF_P + 2 * PB;
    static constexpr int OFF_QS = OFF_RAW + TC_STAGES * STAGE;  // float [2][N]: sums of q
    // of each group's rows:
    static constexpr int OFF_REF = OFF_QS + 2 * N * 4;          // float [2][NC]: minus the reference, 0 when none
    static constexpr int OFF_SET = OFF_REF + 2 * NC * 4;        // float [2][NC]: the reference, -inf when none
    static constexpr int OFF_FAC = OFF_SET + 2 * NC * 4;        // float [2][NC]: a moved reference's factor
    static constexpr int OFF_DEL = OFF_FAC + 2 * NC * 4;        // float [2][NC]: sums of p * zero
    static constexpr int OFF_RED = OFF_DEL + 2 * NC * 4;        // float2 [4 warps][2][NC]
    static constexpr int OFF_AT = OFF_RED + 4 * 2 * NC * 8;     // int64 [N]: output rows
    static constexpr int OFF_MASK = OFF_AT + N * 8;             // uint32 [2][NC][TC_MASK_WORDS]
    static constexpr int OFF_ODD = OFF_MASK + 2 * NC * TC_MASK_WORDS * 4;  // uint32 [2][4 warps][TC_MASK_WORDS]
    static constexpr int OFF_BAD = OFF_ODD + 8 * TC_MASK_WORDS * 4;        // int [TC_STAGES]
    static constexpr int OFF_FLAG = OFF_BAD + TC_STAGES * 4;               // int [2 groups]: a reference has to move
    static constexpr int OFF_BAR = (OFF_FLAG + 8 + 15) / 16 * 16;
    static constexpr int BARS = 2 * TC_STAGES + 17 + SR + 2;
    static constexpr int USED = OFF_BAR + BARS * 8 + 16 + 1024;  // + tensor-memory address, error flag; alignment
    // all of tensor memory is allocated, so no second CTA may fit beside this one
    static constexpr int BYTES = USED > 117 * 1024 ? USED : 117 * 1024;
    static_assert(BYTES <= 227 * 1024, "fits an SM");
    static_assert(2 * (BYTES + 1024) > 228 * 1024, "one CTA an SM");
    // tensor memory columns
    static constexpr int T_K = 0;                  // 2 x D / 2
    static constexpr int T_V = T_K + 2 * (D / 2);  // 2 x 64
    static constexpr int T_S = T_V + 2 * 64;       // SR x N
    static constexpr int T_O = T_S + SR * N;       // ACC x N
    static_assert(T_O + ACC * N <= 512, "tensor memory");
};

// Sums 8 values over the lanes: lane l ends with the sum of value
// 4 b0 + 2 b1 + b2 (b the bits of l).
__device__ __forceinline__ float tc_sum8(const float* v, int lane) {
    float a[4], b[2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float keep = (lane & 1) ? v[4 + i] : v[i], give = (lane & 1) ? v[i] : v[4 + i];
        a[i] = keep + __shfl_xor_sync(0xffffffffu, give, 1);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float keep = (lane & 2) ? a[2 + i] : a[i], give = (lane & 2) ? a[i] : a[2 + i];
        b[i] = keep + __shfl_xor_sync(0xffffffffu, give, 2);
    }
    const float keep = (lane & 4) ? b[1] : b[0], give = (lane & 4) ? b[0] : b[1];
    float s = keep + __shfl_xor_sync(0xffffffffu, give, 4);
    s += __shfl_xor_sync(0xffffffffu, s, 8);
    return s + __shfl_xor_sync(0xffffffffu, s, 16);
}

template <int DT, int D, int N_, bool ALT_>
__global__ void __launch_bounds__(TC_NT, 1) sc_attend_tc_kernel(const __grid_constant__ AttendParams P) {
    using Ty = SC<DT>;
    using Sm = TcShape<DT, D, N_, ALT_>;
    using T = typename Ty::T;
    constexpr int N = Sm::N, NC = Sm::NC;
    constexpr bool ALT = Sm::ALT;
    constexpr unsigned ALL = 0xffffffffu;
    extern __shared__ __align__(1024) unsigned char tc_raw[];
    unsigned char* base = tc_raw + ((1024u - (smem_u32(tc_raw) & 1023u)) & 1023u);
    float* qs_s = reinterpret_cast<float*>(base + Sm::OFF_QS);
    volatile int* bad_s = reinterpret_cast<int*>(base + Sm::OFF_BAD);
    uint32_t* odd_s = reinterpret_cast<uint32_t*>(base + Sm::OFF_ODD);
    volatile int* flag_s = reinterpret_cast<int*>(base + Sm::OFF_FLAG);
    uint64_t* raw_full = reinterpret_cast<uint64_t*>(base + Sm::OFF_BAR);
    uint64_t* raw_empty = raw_full + TC_STAGES;
    uint64_t* ak_full = raw_empty + TC_STAGES;  // expanded keys in tensor memory
    uint64_t* ak_empty = ak_full + 2;
    uint64_t* av_full = ak_empty + 2;           // expanded values
    uint64_t* s_full = av_full + 2;             // scores
    uint64_t* vote = s_full + Sm::SR;           // a softmax group's warps have looked at a tile's scores
    uint64_t* p_full = vote + 2;              // weights stored, scores read
    uint64_t* pv_done = p_full + 2;             // frees the weights and the expanded values
    uint64_t* q_full = pv_done + 2;             // a segment's queries
    uint64_t* q_empty = q_full + 2;
    uint64_t* odd_full = q_empty + 2;           // the scored positions' values have been looked at
    uint64_t* done = odd_full + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
    volatile int* err_s = reinterpret_cast<volatile int*>(tmem_slot + 1);

    // (the broadcast tells the compiler that a role is a whole warp's)
    const int tid = threadIdx.x, warp = __shfl_sync(ALL, tid >> 5, 0), lane = tid & 31;
    const int r8 = lane >> 2, q4 = lane & 3;
    const CacheView& c = P.c;

    pdl_launch_dependents();
    const Range R = sc_range<TC_NT, TC_TILE>(P, TC_MIN_TILES);
    if (tid == 0 && !P.whole) P.desc[blockIdx.x] = make_int4(-1, 0, 0, 0);
    if (R.g0 >= R.g1) return;
    if (tid == 0) {
#pragma unroll 1
        for (int i = 0; i < TC_STAGES; ++i) {
            mbar_init(&raw_full[i], 1);
            mbar_init(&raw_empty[i], 8 + Sm::GROUP_WARPS);
        }
#pragma unroll 1
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ak_full[i], 4);
            mbar_init(&ak_empty[i], 1);
            mbar_init(&av_full[i], 4);
            mbar_init(&vote[i], 4);
            mbar_init(&p_full[i], Sm::GROUP_WARPS);
            mbar_init(&pv_done[i], 1);
            mbar_init(&q_full[i], 4);
            mbar_init(&q_empty[i], 8);
            mbar_init(&odd_full[i], 4);
        }
#pragma unroll 1
        for (int i = 0; i < Sm::SR; ++i) mbar_init(&s_full[i], 1);
        mbar_init(done, 1);
        fence_mbar_init();
        *err_s = 0;
        flag_s[0] = flag_s[1] = 0;
    }
    if (warp == 17) {
        tc_alloc(tmem_slot, 512);
        tc_relinquish();
    }
    tc_before();
    __syncthreads();
    tc_after();
    const uint32_t tmem = *tmem_slot;
    bool failed = false;

    const int nb = TC_TILE >> c.log2_block;  // blocks of a tile
    const uint32_t bbytes = 2 * sc_half_bytes<D>(c.block);
    const uint32_t bstride = bbytes + (c.block == 64 ? 0 : c.block == 32 ? 64 : 32);

    Walk<TC_TILE> w;
    w.begin(P, R);
    const int chunk = static_cast<int>(R.chunk);
    int it = 0;    // tiles so far: buffer it & 1
    int ir = 0;    // cache tiles so far: stage ir % TC_STAGES
    int seg = 0;   // parts with tiles so far: query buffer seg & 1
    int dseg = 0;  // of them, parts with scored positions
    auto cached = [&](int u) { return u * TC_TILE < w.len; };
    auto active = [&]() { return w.len > 0 || P.k_new != nullptr; };

    if (warp >= 16) regs_down<56>();
    if (warp == 16) {
        // ---- the copies ----
        unsigned char* raw = base + Sm::OFF_RAW;
        auto page = [&](int u, int* sub) {  // lane j: block j of tile u
            const int t = u * TC_TILE + (lane << c.log2_block);
            *sub = (t & (c.page_size - 1)) >> c.log2_block;
            return (lane < nb && t < w.len)
                       ? __ldg(c.table + static_cast<size_t>(w.b) * c.max_pages + (t >> c.log2_page))
                       : -2;
        };
#pragma unroll 1
        for (bool go = true; go && !failed; go = w.next(P)) {
            const int head = w.hr / P.row_blocks;
            int sub, id = page(w.u0, &sub);
#pragma unroll 1
            for (int u = w.u0; u < w.u1 && cached(u); ++u) {
                const int s = ir % TC_STAGES;
                if (ir >= TC_STAGES &&
                    !sc_wait(&raw_empty[s], ((ir / TC_STAGES) - 1) & 1, P.timeout_ns)) {
                    failed = true;
                    break;
                }
                const bool mine = id != -2;
                const bool ok = mine && id >= 0 && id < c.num_pages && !P.test_hook;
                const unsigned got = __ballot_sync(ALL, ok), want = __ballot_sync(ALL, mine);
                if (lane == 0) {
                    bad_s[s] = got != want && !P.test_hook;
                    mbar_arrive_expect_tx(&raw_full[s], P.test_hook ? bbytes : bbytes * __popc(got));
                }
                __syncwarp();
                if (ok)
                    bulk_g2s(raw + s * Sm::STAGE + lane * bstride, sc_block_ptr<D>(c, id, head, sub), bbytes, &raw_full[s]);
                ++ir;
                id = page(u + 1, &sub);
            }
        }
        // no copy may land after the CTA is gone
#pragma unroll 1
        for (int i = ir > TC_STAGES ? ir - TC_STAGES : 0; i < ir; ++i)
            if (!sc_wait(&raw_full[i % TC_STAGES], (i / TC_STAGES) & 1, P.timeout_ns)) failed = true;
    } else if (warp == 17) {
        // ---- the MMAs: whichever product has its operands, O first; the warp stays
        // together and one elected lane issues, so that the operands are uniform ----
        constexpr uint32_t id_qk = tc_idesc(DT == 0, N), id_pv = tc_idesc(1, N);
        const bool leader = sc_elect();
        const uint64_t q_desc = tc_desc(smem_u32(base)), p_desc = tc_desc(smem_u32(base + Sm::OFF_P));
        int qi = 0, pi = 0;              // the next tile's S, and O
        uint32_t firsts = 0, denses = 0;  // bit i & 31: of tile i
        bool more = true;                // tiles left to score
        while (more && !active()) more = w.next(P);
        int u = w.u0;
        uint64_t t0 = 0;
        uint32_t idle = 0;
#pragma unroll 1
        while ((more || pi < qi) && !failed) {
            bool did = false;
            if (pi < qi && tc_test(&p_full[pi & 1], (pi >> 1) & 1) && tc_test(&av_full[pi & 1], (pi >> 1) & 1)) {
                const int b = pi & 1;
                const bool dense = (denses >> (pi & 31)) & 1u, first = (firsts >> (pi & 31)) & 1u;
                tc_after();
                if (leader) {
                    const uint32_t a = tmem + Sm::T_V + b * 64, o = tmem + Sm::T_O + (ALT ? b * N : 0);
                    const uint64_t pd = p_desc + static_cast<uint64_t>(b * (Sm::PB >> 4));
                    // with fp16 activations the scored positions keep their type; the codes are
                    // bf16, and their weights come in two parts
                    const uint32_t idesc = DT == 1 && dense ? id_qk : id_pv;
                    const int parts = DT == 1 && dense ? 1 : Sm::PSPLIT;
#pragma unroll 1
                    for (int part = 0; part < parts; ++part)
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            tc_mma(o, a + 8 * k, pd + (part * 2 * Sm::HALF + (k >> 2) * Sm::HALF + (k & 3) * 32) / 16, idesc,
                                   (first && part == 0 && k == 0) ? 0u : 1u);
                    tc_commit(&pv_done[b]);
                }
                __syncwarp();
                ++pi;
                did = true;
            }
            // (the scores of tile qi - SR have been read once its weights are there)
            if (more && qi - pi < Sm::SR && tc_test(&ak_full[qi & 1], (qi >> 1) & 1)) {
                const int b = qi & 1;
                tc_after();
                if (leader) {
                    const uint64_t qd = q_desc + static_cast<uint64_t>((seg & 1) * (Sm::Q >> 4));
#pragma unroll
                    for (int k = 0; k < D / 16; ++k)
                        tc_mma(tmem + Sm::T_S + (qi % Sm::SR) * N, tmem + Sm::T_K + b * (D / 2) + 8 * k,
                               qd + ((k >> 2) * Sm::HALF + (k & 3) * 32) / 16, id_qk, k != 0);
                    tc_commit(&ak_empty[b]);
                    tc_commit(&s_full[qi % Sm::SR]);
                }
                __syncwarp();
                const uint32_t bit = 1u << (qi & 31);
                firsts = u - w.u0 < Sm::ACC ? firsts | bit : firsts & ~bit;
                denses = cached(u) ? denses & ~bit : denses | bit;
                ++qi;
                if (++u == w.u1) {
                    ++seg;
                    do more = w.next(P);
                    while (more && !active());
                    u = w.u0;
                }
                did = true;
            }
            if (did) {
                idle = 0;
            } else {
                __nanosleep(64);
                if ((++idle & 63u) == 0u) {  // nothing for a while: mind the clock
                    const uint64_t now = globaltimer_ns();
                    if (idle == 64u) t0 = now;
                    if (now - t0 > P.timeout_ns) failed = true;
                }
                failed = __any_sync(ALL, failed);
            }
        }
        if (leader) tc_commit(done);
    } else if (warp < 4) {
        regs_down<72>();
        // ---- keys: queries of a segment, then codes to tensor memory ----
        // a lane's tokens are 32 warp + 8 i + r8; its bytes of tokens i = 0 and 2 (1 and 3 lie 8 rows on)
        uint32_t off[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int t = 32 * warp + 16 * i + r8;
            off[i] = (t >> c.log2_block) * bstride + (t & (c.block - 1)) * (D / 2) + q4 * (D / 8);
        }
#pragma unroll 1
        for (bool go = true; go && !failed; go = w.next(P)) {
            if (!active()) continue;
            const int head = w.hr / P.row_blocks, row0 = (w.hr % P.row_blocks) * N, qb = seg & 1;
            if (seg >= 2 && !sc_wait(&q_empty[qb], ((seg >> 1) - 1) & 1, P.timeout_ns)) {
                failed = true;
                break;
            }
            // column 8 j + 2 q + e of the key operand holds the dims (D / 4) q + 4 j + 2 e, + 1:
            // the queries take the same order
#pragma unroll 1
            for (int i = tid; i < N * (D / 8); i += 128) {
                const int r = i / (D / 8), ch = i % (D / 8), row = row0 + r;
                uint4 x = make_uint4(0u, 0u, 0u, 0u);
                if (row < P.rows) {
                    const int node = row / P.group, g = row - node * P.group;
                    const T* src = static_cast<const T*>(P.q) + (static_cast<long long>(w.b) * P.n + node) * P.q_stride +
                                   static_cast<long long>(head * P.group + g) * D + (D / 2) * (ch & 1) + 4 * (ch >> 1);
                    const uint2 lo = *reinterpret_cast<const uint2*>(src), hi = *reinterpret_cast<const uint2*>(src + D / 4);
                    x = make_uint4(lo.x, lo.y, hi.x, hi.y);
                    if constexpr (DT == 0) {  // 2^64, and 2^60 where the code is 16-fold (exact)
                        x.x = Ty::pack(Ty::lo(x.x) * SC_2P64, Ty::hi(x.x) * SC_2P64);
                        x.y = Ty::pack(Ty::lo(x.y) * SC_2P60, Ty::hi(x.y) * SC_2P60);
                        x.z = Ty::pack(Ty::lo(x.z) * SC_2P64, Ty::hi(x.z) * SC_2P64);
                        x.w = Ty::pack(Ty::lo(x.w) * SC_2P60, Ty::hi(x.w) * SC_2P60);
                    }
                }
                *reinterpret_cast<uint4*>(base + qb * Sm::Q + (ch >> 3) * Sm::HALF + r * 128 + (((ch & 7) ^ (r & 7)) << 4)) = x;
            }
            if (tid < N) {
                const int row = row0 + tid;
                float s = 0.f;
                if (row < P.rows) {
                    const int node = row / P.group, g = row - node * P.group;
                    const T* src = static_cast<const T*>(P.q) + (static_cast<long long>(w.b) * P.n + node) * P.q_stride +
                                   static_cast<long long>(head * P.group + g) * D;
#pragma unroll 4
                    for (int k = 0; k < D / 8; ++k) {
                        const uint4 x = *reinterpret_cast<const uint4*>(src + 8 * k);
                        s += (Ty::lo(x.x) + Ty::hi(x.x)) + (Ty::lo(x.y) + Ty::hi(x.y)) + (Ty::lo(x.z) + Ty::hi(x.z)) +
                             (Ty::lo(x.w) + Ty::hi(x.w));
                    }
                }
                qs_s[qb * N + tid] = s;
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) sc_arrive(&q_full[qb]);
            int u = w.u0;
            const int uc = min(w.u1, (w.len + TC_TILE - 1) / TC_TILE);  // behind the cache tiles
#pragma unroll 1
            for (; u < uc; ++u, ++it, ++ir) {
                const int b = it & 1;
                if (!(it < 2 || sc_wait(&ak_empty[b], ((it >> 1) - 1) & 1, P.timeout_ns)) ||
                    !sc_wait(&raw_full[ir % TC_STAGES], (ir / TC_STAGES) & 1, P.timeout_ns)) {
                    failed = true;
                    break;
                }
                tc_after();
                const uint32_t dst = tmem + Sm::T_K + b * (D / 2) + (static_cast<uint32_t>(32 * warp) << 16);
                const unsigned char* tile = base + Sm::OFF_RAW + (ir % TC_STAGES) * Sm::STAGE;
                uint32_t kw[4][D / 32];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const unsigned char* a = tile + off[i >> 1] + (i & 1) * 8 * (D / 2);
                    if constexpr (D == 128) {
                        const uint4 v = *reinterpret_cast<const uint4*>(a);
                        kw[i][0] = v.x, kw[i][1] = v.y, kw[i][2] = v.z, kw[i][3] = v.w;
                    } else {
                        const uint2 v = *reinterpret_cast<const uint2*>(a);
                        kw[i][0] = v.x, kw[i][1] = v.y;
                    }
                }
#pragma unroll
                for (int h2 = 0; h2 < 2; ++h2)
#pragma unroll
                    for (int s = 0; s < D / 64; ++s) {
                        uint32_t x[16];
#pragma unroll
                        for (int k = 0; k < 2; ++k)
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                const uint32_t wd = kw[2 * h2 + y][2 * s + k], w8 = wd >> 8;
#pragma unroll
                                for (int j = 0; j < 4; ++j)
                                    x[8 * k + 4 * (j >> 1) + 2 * y + (j & 1)] = sc_codes<DT == 0>(wd, w8, j);
                            }
                        tc_st16(dst + (static_cast<uint32_t>(16 * h2) << 16) + 32 * s, x);
                    }
                tc_wait_st();
                tc_before();
                __syncwarp();
                if (lane == 0) {
                    sc_arrive(&raw_empty[ir % TC_STAGES]);
                    sc_arrive(&ak_full[b]);
                }
            }
#pragma unroll 1
            for (; u < w.u1 && !failed; ++u, ++it) {
                const int b = it & 1;
                if (it >= 2 && !sc_wait(&ak_empty[b], ((it >> 1) - 1) & 1, P.timeout_ns)) {
                    failed = true;
                    break;
                }
                tc_after();
                const uint32_t dst = tmem + Sm::T_K + b * (D / 2) + (static_cast<uint32_t>(32 * warp) << 16);
                const int j0 = (u - (w.len + TC_TILE - 1) / TC_TILE) * TC_TILE;
#pragma unroll 1
                for (int hs = 0; hs < 2 * (D / 64); ++hs) {
                    const int h2 = hs / (D / 64), s = hs % (D / 64);
                    uint32_t x[16];
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const int j = j0 + 32 * warp + 16 * h2 + 8 * y + r8;
                        const T* src = static_cast<const T*>(P.k_new) + (static_cast<long long>(w.b) * P.n + j) * P.kv_stride +
                                       static_cast<long long>(head) * D + q4 * (D / 4) + 16 * s;
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            uint4 v = j < P.n ? *reinterpret_cast<const uint4*>(src + 8 * i) : make_uint4(0u, 0u, 0u, 0u);
                            if constexpr (DT == 0) {  // against the queries' 2^60
                                v.y = Ty::pack(Ty::lo(v.y) * 16.f, Ty::hi(v.y) * 16.f);
                                v.w = Ty::pack(Ty::lo(v.w) * 16.f, Ty::hi(v.w) * 16.f);
                            }
                            x[8 * i + 2 * y] = v.x, x[8 * i + 2 * y + 1] = v.y;
                            x[8 * i + 4 + 2 * y] = v.z, x[8 * i + 4 + 2 * y + 1] = v.w;
                        }
                    }
                    __syncwarp();
                    tc_st16(dst + (static_cast<uint32_t>(16 * h2) << 16) + 32 * s, x);
                }
                tc_wait_st();
                tc_before();
                __syncwarp();
                if (lane == 0) sc_arrive(&ak_full[b]);
            }
            ++seg;
        }
    } else if (warp < 8) {
        regs_down<72>();
        // ---- values: codes to tensor memory, a lane of it a dim ----
        const int wq = warp & 3;
        uint32_t off[2];  // this lane's 16 tokens of each 64, in the rows of dim 32 wq + r8
#pragma unroll
        for (int hb = 0; hb < 2; ++hb) {
            const int tq = 64 * hb + 16 * q4;
            off[hb] = (tq >> c.log2_block) * bstride + sc_half_bytes<D>(c.block) + (tq & (c.block - 1)) / 2 +
                      (32 * wq + r8) * (c.block / 2);
        }
        const uint32_t rows8 = 8 * (c.block / 2);
#pragma unroll 1
        for (bool go = true; go && !failed; go = w.next(P)) {
            if (!active()) continue;
            const int head = w.hr / P.row_blocks;
            if (seg >= 2 && !sc_wait(&q_empty[seg & 1], ((seg >> 1) - 1) & 1, P.timeout_ns)) {
                failed = true;
                break;
            }
            int u = w.u0;
            const int uc = min(w.u1, (w.len + TC_TILE - 1) / TC_TILE);
#pragma unroll 1
            for (; u < uc; ++u, ++it, ++ir) {
                const int b = it & 1;
                if (!(it < 2 || sc_wait(&pv_done[b], ((it >> 1) - 1) & 1, P.timeout_ns)) ||
                    !sc_wait(&raw_full[ir % TC_STAGES], (ir / TC_STAGES) & 1, P.timeout_ns)) {
                    failed = true;
                    break;
                }
                tc_after();
                if (32 * wq < D) {
                    const uint32_t dst = tmem + Sm::T_V + b * 64 + (static_cast<uint32_t>(32 * wq) << 16);
                    const unsigned char* tile = base + Sm::OFF_RAW + (ir % TC_STAGES) * Sm::STAGE;
                    uint2 v[2][4];
#pragma unroll
                    for (int hb = 0; hb < 2; ++hb)
#pragma unroll
                        for (int i = 0; i < 4; ++i) v[hb][i] = *reinterpret_cast<const uint2*>(tile + off[hb] + i * rows8);
#pragma unroll
                    for (int hb = 0; hb < 2; ++hb)
#pragma unroll
                        for (int h2 = 0; h2 < 2; ++h2) {
                            uint32_t x[16];
#pragma unroll
                            for (int k = 0; k < 2; ++k)
#pragma unroll
                                for (int y = 0; y < 2; ++y) {
                                    const uint32_t wd = k ? v[hb][2 * h2 + y].y : v[hb][2 * h2 + y].x, w8 = wd >> 8;
#pragma unroll
                                    for (int j = 0; j < 4; ++j)
                                        x[8 * k + 4 * (j >> 1) + 2 * y + (j & 1)] =
                                            DT == 0 ? sc_codes<true>(wd, w8, j) : sc_center_bf16(sc_codes_bf16(wd, j));
                                }
                            tc_st16(dst + (static_cast<uint32_t>(16 * h2) << 16) + 32 * hb, x);
                        }
                    tc_wait_st();
                }
                tc_before();
                __syncwarp();
                if (lane == 0) {
                    sc_arrive(&raw_empty[ir % TC_STAGES]);
                    sc_arrive(&av_full[b]);
                }
            }
            const bool dense = u < w.u1;
            // the scored positions' own values; an element that is not finite is left out of
            // the product, where it would reach the rows that do not see it, and noted
            uint32_t* odd = odd_s + ((dseg & 1) * 4 + wq) * TC_MASK_WORDS;
            if (dense && lane < TC_MASK_WORDS) odd[lane] = 0u;
#pragma unroll 1
            for (; u < w.u1 && !failed; ++u, ++it) {
                const int b = it & 1;
                if (it >= 2 && !sc_wait(&pv_done[b], ((it >> 1) - 1) & 1, P.timeout_ns)) {
                    failed = true;
                    break;
                }
                tc_after();
                __syncwarp();
                const uint32_t dst = tmem + Sm::T_V + b * 64 + (static_cast<uint32_t>(32 * wq) << 16);
                const int j0 = (u - (w.len + TC_TILE - 1) / TC_TILE) * TC_TILE;
                if (32 * wq < D) {
#pragma unroll 1
                    for (int hh = 0; hh < 4; ++hh) {
                        const int hb = hh >> 1, h2 = hh & 1;
                        uint32_t x[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) x[i] = 0u;
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const int j1 = j0 + 64 * hb + 16 * q4;  // this lane's 16 positions
                            const uint16_t* src = static_cast<const uint16_t*>(P.v_new) +
                                                  (static_cast<long long>(w.b) * P.n + j1) * P.kv_stride +
                                                  static_cast<long long>(head) * D + 32 * wq + 16 * h2 + 8 * y + r8;
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                uint32_t e = j1 + i < P.n ? src[i * P.kv_stride] : 0u;
                                if (!(fabsf(Ty::lo(e)) < __builtin_huge_valf())) {
                                    atomicOr(&odd[(j1 + i) >> 5], 1u << ((j1 + i) & 31));
                                    e = 0u;
                                }
                                x[4 * (i >> 2) + 2 * y + ((i >> 1) & 1)] |= e << (16 * (i & 1));
                            }
                        }
                        __syncwarp();
                        tc_st16(dst + (static_cast<uint32_t>(16 * h2) << 16) + 32 * hb, x);
                    }
                }
                tc_wait_st();
                tc_before();
                __syncwarp();
                if (lane == 0) sc_arrive(&av_full[b]);
            }
            if (dense) {
                __syncwarp();
                if (lane == 0 && !failed) sc_arrive(&odd_full[dseg & 1]);
                ++dseg;
            }
            ++seg;
        }
    } else if (warp < 16) {
        regs_up<136>();
        // ---- softmax: thread = token, NC rows ----
        const int half = (warp - 8) >> 2, wq = warp & 3, tt = tid - 256 - half * 128;
        const int col0 = ALT ? 0 : half * NC, bar = 1 + half;
        float* ref_s = reinterpret_cast<float*>(base + Sm::OFF_REF) + half * NC;
        float* set_s = reinterpret_cast<float*>(base + Sm::OFF_SET) + half * NC;
        float* fac_s = reinterpret_cast<float*>(base + Sm::OFF_FAC) + half * NC;
        float2* red_s = reinterpret_cast<float2*>(base + Sm::OFF_RED) + half * NC;
        constexpr int RS = 2 * NC;  // of red_s, from warp to warp
        uint32_t* mask_s = reinterpret_cast<uint32_t*>(base + Sm::OFF_MASK) + half * NC * TC_MASK_WORDS;
        const uint32_t lane_base = static_cast<uint32_t>(32 * wq) << 16;
        const uint32_t o_addr = tmem + Sm::T_O + (ALT ? half * N : col0) + lane_base;
        const bool o_mine = 32 * wq < D;
        const int t = 32 * wq + lane;
        // place of token t in the weights' K order: k = 16 ((t % 16) / 4) + 4 ((t % 64) / 16) + t % 4
        const int kk = 16 * ((t & 15) >> 2) + 4 * ((t & 63) >> 4) + (t & 3);
        const uint32_t kx = static_cast<uint32_t>(((kk >> 3) << 4) | ((kk & 7) * 2));
        const uint32_t poff = (t >> c.log2_block) * bstride + c.block * (D / 2) + (t & (c.block - 1)) * 4;
        const float sl = P.scale * SC_LOG2E;
        const float nan = __int_as_float(0x7fffffff);
        // what a code's product, a scored position's product and a weight are multiplied by
        const float k_code = DT == 0 ? SC_2P69 : 16777216.f;
        const float k_new = DT == 0 ? 1.f / SC_2P64 : 1.f;
        const float v_code = DT == 0 ? ((t & 2) ? SC_2P60 : SC_2P64) : 1.f;
        const float v_off = -8.f / v_code;
        const float v_new = DT == 0 ? 1.f / SC_2P69 : 1.f;
        const float o_scale = DT == 0 ? SC_2P69 : 1.f;
        uint32_t votes = 0;

#pragma unroll 1
        for (bool go = true; go; go = w.next(P)) {
            const int head = w.hr / P.row_blocks, row0 = (w.hr % P.row_blocks) * N + col0;  // this thread's first row
            uint64_t l[NC / 2], z[NC / 2];
#pragma unroll
            for (int i = 0; i < NC / 2; ++i) l[i] = z[i] = 0ull;
            auto poison = [&]() {
#pragma unroll
                for (int i = 0; i < NC / 2; ++i) l[i] = 0x7fffffff7fffffffull;
            };
            if (w.bad) poison();
            if (tt < NC) {
                ref_s[tt] = 0.f;
                set_s[tt] = SC_NEG_INF;
            }
            named_sync(bar, 128);
            const bool act = active();
            bool unset = true, fresh = true, dense = false;  // a row without reference; no weights yet; scored positions
            if (act && !failed && !sc_wait(&q_full[seg & 1], (seg >> 1) & 1, P.timeout_ns)) failed = true;
            const int it0 = it;
            const int tiles = act ? w.u1 - w.u0 : 0;
            const float* qs = qs_s + (seg & 1) * N + col0;
#pragma unroll 1
            for (int u = w.u0; u < w.u0 + tiles; ++u, ++it) {
                const bool code = cached(u);
                const int stage = ir % TC_STAGES;
                const uint32_t raw_phase = (ir / TC_STAGES) & 1;
                if (code) {
                    ++ir;
                } else if (!dense) {  // scored positions: who sees whom, for these rows
                    dense = true;
                    const int32_t* par = P.parents ? P.parents + static_cast<size_t>(w.b) * (P.n - 1) : nullptr;
                    int wrong = 0;
                    if (par)
#pragma unroll 1
                        for (int i = 1 + tt; i < P.n; i += 128) wrong |= par[i - 1] < 0 || par[i - 1] >= i;
                    const bool no_tree = named_or(bar, 128, wrong != 0);
                    if (no_tree) poison();
                    if (tt < NC) {
                        uint32_t* m = mask_s + tt * TC_MASK_WORDS;
                        const int row = row0 + tt, node = row / P.group;
                        const bool all = !par || no_tree || row >= P.rows;
                        // rows behind the last see everything; without parents node i sees 0 .. i
                        const int hi = row < P.rows ? node : P.n;
#pragma unroll 1
                        for (int i = 0; i < TC_MASK_WORDS; ++i)
                            m[i] = !all || i * 32 > hi ? 0u : hi - i * 32 >= 31 ? ALL : (2u << (hi - i * 32)) - 1u;
                        if (!all)
#pragma unroll 1
                            for (int a = node;; a = par[a - 1]) {
                                m[a >> 5] |= 1u << (a & 31);
                                if (a == 0) break;
                            }
                    }
                    named_sync(bar, 128);
                }
                const int b = it & 1, sb = it % Sm::SR;
                if (ALT && b != half) continue;
                float ka = sl * k_new, kb = 0.f, vs = v_new, vz = 0.f, off = 0.f;
                int valid, j0 = 0;  // tokens of the tile; its first scored position
                if (code) {
                    valid = w.len - u * TC_TILE;
                    if (!failed && !sc_wait(&raw_full[stage], raw_phase, P.timeout_ns)) failed = true;
                    const unsigned char* par = base + Sm::OFF_RAW + stage * Sm::STAGE + poff;
                    const uint32_t kp = *reinterpret_cast<const uint32_t*>(par);
                    const uint32_t vp = *reinterpret_cast<const uint32_t*>(par + sc_half_bytes<D>(c.block));
                    const bool bad = __any_sync(ALL, bad_s[stage]);
                    __syncwarp();
                    if (lane == 0) sc_arrive(&raw_empty[stage]);
                    if (bad) poison();
                    ka = Ty::lo(kp) * sl * k_code;
                    kb = Ty::hi(kp) * sl;
                    vs = Ty::lo(vp);
                    vz = fmaf(8.f, vs, Ty::hi(vp));  // the values' middle: codes count from 8
                    vs *= v_code;
                    off = v_off;
                    if (t >= valid) ka = kb = vs = vz = 0.f;
                } else {
                    j0 = (u - (w.len + TC_TILE - 1) / TC_TILE) * TC_TILE;
                    valid = P.n - j0;
                }
                if (!failed && !sc_wait(&s_full[sb], (it / Sm::SR) & 1, P.timeout_ns)) failed = true;
                __syncwarp();
                tc_after();
                const uint32_t s_addr = tmem + Sm::T_S + sb * N + col0 + lane_base;
                const uint64_t a2 = f2_pack(ka, ka), b2 = f2_pack(kb, kb);
                const bool special = !code || valid < TC_TILE;
                // scores of 8 rows relative to the reference: scale (q . code) + zero sum(q) - reference
                auto relative = [&](float* d, int i0) {
#pragma unroll
                    for (int i = 0; i < 8; i += 4) {
                        const ulonglong2 q2 = *reinterpret_cast<const ulonglong2*>(qs + i0 + i);
                        const ulonglong2 n2 = *reinterpret_cast<const ulonglong2*>(ref_s + i0 + i);
                        const uint64_t x = f2_fma(a2, f2_pack(d[i], d[i + 1]), f2_fma(b2, q2.x, n2.x));
                        const uint64_t y = f2_fma(a2, f2_pack(d[i + 2], d[i + 3]), f2_fma(b2, q2.y, n2.y));
                        f2_unpack(x, d[i], d[i + 1]);
                        f2_unpack(y, d[i + 2], d[i + 3]);
                    }
                    if (special) {  // the last cache tile, and scored positions
                        const uint32_t* m = mask_s + i0 * TC_MASK_WORDS + (j0 >> 5) + wq;
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (t >= valid || (!code && !((m[i * TC_MASK_WORDS] >> lane) & 1u))) d[i] = SC_NEG_INF;
                    }
                };
                float p[NC];
#pragma unroll 1
                for (bool moved = false;; moved = true) {
#pragma unroll
                    for (int g = 0; g < NC; g += 8) tc_ld8(s_addr + g, *reinterpret_cast<float(*)[8]>(p + g));
                    tc_wait_ld();
                    float top = SC_NEG_INF;
#pragma unroll
                    for (int g = 0; g < NC; g += 8) {
                        relative(p + g, g);
#pragma unroll
                        for (int i = 0; i < 8; ++i) top = fmaxf(top, p[g + i]);
                    }
                    // the group's warps vote whether a reference has to move, and go on meanwhile
                    if (__any_sync(ALL, top > 8.f || failed) && lane == 0) flag_s[half] = 1;
                    __syncwarp();
                    if (lane == 0) sc_arrive(&vote[half]);
#pragma unroll
                    for (int i = 0; i < NC; ++i) p[i] = ex2(p[i]);
                    // the weights' buffer, and the accumulator a moved reference rescales, are free
                    // when this group's (the tile before last's) product is done
                    if (it >= 2 && !failed && !sc_wait(&pv_done[b], ((it >> 1) - 1) & 1, P.timeout_ns)) failed = true;
                    // the slowest of the four warps may first have waited for its scores in vain
                    if (!sc_wait(&vote[half], votes & 1, 4 * P.timeout_ns)) failed = true;
                    ++votes;
                    if (moved || !(__any_sync(ALL, flag_s[half]) || unset)) break;
                    // ---- move the references that have none, or that a score passed by 2^8, and
                    // look at the tile again (its scores are still in tensor memory) ----
                    if (named_or(bar, 128, failed)) failed = true;
#pragma unroll 1
                    for (int g = 0; g < NC; g += 8) {
                        float x[8];
                        tc_ld8(s_addr + g, x);
                        tc_wait_ld();
                        relative(x, g);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            x[i] = warp_max_f32(x[i]);
                            if (lane == 0) red_s[wq * RS + g + i].x = x[i];
                        }
                    }
                    named_sync(bar, 128);
                    if (tt == 0) flag_s[half] = 0;
                    if (tt < NC) {
                        const float md = fmaxf(fmaxf(red_s[tt].x, red_s[RS + tt].x),
                                               fmaxf(red_s[2 * RS + tt].x, red_s[3 * RS + tt].x));
                        const float old = set_s[tt], x = md - ref_s[tt];
                        float f = 1.f;
                        if (x > old + 8.f) {
                            f = old == SC_NEG_INF ? 0.f : ex2(old - x);
                            set_s[tt] = x;
                            ref_s[tt] = -x;
                        }
                        fac_s[tt] = f;
                    }
                    unset = named_or(bar, 128, tt < NC && set_s[tt < NC ? tt : 0] == SC_NEG_INF);
                    if (fresh) continue;
#pragma unroll
                    for (int i = 0; i < NC; i += 2) {
                        const uint64_t f = *reinterpret_cast<const uint64_t*>(fac_s + i);
                        l[i / 2] = f2_mul(l[i / 2], f);
                        z[i / 2] = f2_mul(z[i / 2], f);
                    }
                    if (!failed && !ALT && !sc_wait(&pv_done[(it - 1) & 1], ((it - 1) >> 1) & 1, P.timeout_ns)) failed = true;
                    tc_after();
                    __syncwarp();
                    if (o_mine && !failed) {
#pragma unroll 1
                        for (int g = 0; g < NC; g += 8) {
                            float x[8];
                            tc_ld8(o_addr + g, x);
                            tc_wait_ld();
#pragma unroll
                            for (int i = 0; i < 8; ++i) x[i] *= fac_s[g + i];
                            tc_st8(o_addr + g, x);
                        }
                        tc_wait_st();
                    }
                }
                // ---- weights ----
                unsigned char* pb = base + Sm::OFF_P + b * Sm::PB + (t >> 6) * Sm::HALF + col0 * 128;
                const uint64_t vs2 = f2_pack(vs, vs), vz2 = f2_pack(vz, vz);
                // bf16 codes count from 0 in the product: 8 of the rounded weight are taken off again,
                // so that a weight's rounding meets code - 8 and not code
                const uint64_t off2 = f2_pack(off, off);
#pragma unroll
                for (int i = 0; i < NC; i += 2) {
                    const uint64_t p2 = f2_pack(p[i], p[i + 1]);
                    l[i / 2] = f2_add(l[i / 2], p2);
                    z[i / 2] = f2_fma(p2, vz2, z[i / 2]);
                    float s0, s1;
                    f2_unpack(f2_mul(p2, vs2), s0, s1);
                    // codes: bf16 whatever the cache's type, since p * scale keeps fp32's range there
                    const uint32_t x = (DT == 0 || code) ? SC<0>::pack(s0, s1) : Ty::pack(s0, s1);
                    if constexpr (DT == 0) z[i / 2] = f2_fma(f2_pack(SC<0>::lo(x), SC<0>::hi(x)), off2, z[i / 2]);
                    unsigned char* e0 = pb + i * 128 + (kx ^ ((i & 7) << 4));
                    unsigned char* e1 = pb + (i + 1) * 128 + (kx ^ (((i + 1) & 7) << 4));
                    *reinterpret_cast<uint16_t*>(e0) = static_cast<uint16_t>(x);
                    *reinterpret_cast<uint16_t*>(e1) = static_cast<uint16_t>(x >> 16);
                    if constexpr (DT == 1) {
                        const uint32_t y = SC<0>::pack(s0 - SC<0>::lo(x), s1 - SC<0>::hi(x));
                        *reinterpret_cast<uint16_t*>(e0 + 2 * Sm::HALF) = static_cast<uint16_t>(y);
                        *reinterpret_cast<uint16_t*>(e1 + 2 * Sm::HALF) = static_cast<uint16_t>(y >> 16);
                    }
                }
                fresh = false;
                fence_async_smem();
                tc_before();
                __syncwarp();
                if (lane == 0) sc_arrive(&p_full[b]);
            }
            // ---- the segment's end: sums over the tokens, the two groups together, the output ----
#pragma unroll 1
            for (int k = 1; k <= 2; ++k)  // the last two products
                if (tiles >= k && !failed && !sc_wait(&pv_done[(it - k) & 1], ((it - k) >> 1) & 1, P.timeout_ns)) failed = true;
            if (dense && !failed && !sc_wait(&odd_full[dseg & 1], (dseg >> 1) & 1, P.timeout_ns)) failed = true;
            tc_after();
#pragma unroll
            for (int g = 0; g < NC / 8; ++g) {
                float a[8], e[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    f2_unpack(l[4 * g + i], a[2 * i], a[2 * i + 1]);
                    f2_unpack(z[4 * g + i], e[2 * i], e[2 * i + 1]);
                }
                const float ls = tc_sum8(a, lane), zs = tc_sum8(e, lane);
                const int i = 8 * g + 4 * (lane & 1) + (lane & 2) + ((lane >> 2) & 1);
                if (lane < 8) red_s[wq * RS + i] = make_float2(ls, zs);
            }
            if (named_or(3, 256, failed)) failed = true;
            const bool whole = w.whole();
            const int slot = blockIdx.x * 2 + (w.u0 == 0 ? 1 : 0);
            constexpr int NO = N / 2;  // rows this group writes
            const int c0 = half * NO;  // the first of them in the block
            float* f_s = reinterpret_cast<float*>(base + Sm::OFF_FAC) + c0;  // [ACC][N]: of the accumulators
            float* z_s = reinterpret_cast<float*>(base + Sm::OFF_DEL) + c0;  // [N]
            long long* at_s = reinterpret_cast<long long*>(base + Sm::OFF_AT) + c0;  // [N]: where a row goes, -1: nowhere
            if (tt < NO) {
                const int col = c0 + tt, row = (w.hr % P.row_blocks) * N + col;
                const float* sets = reinterpret_cast<const float*>(base + Sm::OFF_SET);
                const float2* red = reinterpret_cast<const float2*>(base + Sm::OFF_RED);
                float M = SC_NEG_INF, L = 0.f, Z = 0.f, wt[Sm::ACC];
#pragma unroll
                for (int a = 0; a < Sm::ACC; ++a) M = fmaxf(M, sets[a * NC + col]);
#pragma unroll
                for (int a = 0; a < Sm::ACC; ++a) {
                    float La = 0.f, Za = 0.f;
#pragma unroll 1
                    for (int i = 0; i < 4; ++i) {
                        const float2 v = red[i * RS + a * NC + col];
                        La += v.x;
                        Za += v.y;
                    }
                    const float m = sets[a * NC + col];
                    wt[a] = m == SC_NEG_INF ? 0.f : ex2(m - M);
                    const float f = m == SC_NEG_INF ? 1.f : wt[a];  // (without a reference the sum is 0 or NaN)
                    L = fmaf(La, f, L);
                    Z = fmaf(Za, f, Z);
                }
                if (failed) L = nan;
                // (a sum that is not a number makes its factors one, whatever was accumulated)
                const float norm = L != L ? nan : !whole ? 1.f : L == 0.f ? 0.f : 1.f / L;
#pragma unroll
                for (int a = 0; a < Sm::ACC; ++a) f_s[a * N + tt] = wt[a] * norm * o_scale;
                z_s[tt] = Z * norm;
                long long at = -1;
                if (!whole) {
                    P.part_ml[static_cast<size_t>(slot) * N + col] = make_float2(M, L);
                    at = (static_cast<long long>(slot) * N + col) * D;
                } else if (row < P.rows) {
                    const size_t o = sc_out_row(P, w.b, head, row);
                    if (P.out_lse) P.out_lse[o] = L == 0.f ? SC_NEG_INF : (M + log2f(L)) * SC_LN2;
                    at = static_cast<long long>(o) * D;
                }
                at_s[tt] = at;
            }
            named_sync(bar, 128);
            if (o_mine) {
#pragma unroll 1
                for (int g = 0; g < NO; g += 8) {
                    float x[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] = 0.f;
#pragma unroll 1
                    for (int a = 0; a < Sm::ACC; ++a) {
                        // accumulator a was used by the part's tiles of its turn
                        if (!failed && tiles > 0 && (tiles > 1 || !ALT || (it0 & 1) == a)) {
                            float y[8];
                            tc_ld8(tmem + Sm::T_O + a * N + c0 + g + lane_base, y);
                            tc_wait_ld();
#pragma unroll
                            for (int i = 0; i < 8; ++i) x[i] = fmaf(y[i], f_s[a * N + g + i], x[i]);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] = fmaf(0.f, f_s[g + i], x[i] + z_s[g + i]);
                    if (dense) {
                        const uint32_t* odd = odd_s + ((dseg & 1) * 4 + wq) * TC_MASK_WORDS;  // these 32 dims' warp
                        const uint32_t* mask = reinterpret_cast<const uint32_t*>(base + Sm::OFF_MASK) + (c0 + g) * TC_MASK_WORDS;
#pragma unroll 1
                        for (int wd = 0; wd * 32 < P.n; ++wd)
#pragma unroll 1
                            for (uint32_t m = odd[wd]; m; m &= m - 1) {
                                const int j = wd * 32 + __ffs(m) - 1;
                                const uint16_t e = reinterpret_cast<const uint16_t*>(P.v_new)
                                    [(static_cast<long long>(w.b) * P.n + j) * P.kv_stride + static_cast<long long>(head) * D + t];
                                const float v = Ty::lo(e);
                                if (!(fabsf(v) < __builtin_huge_valf())) {
#pragma unroll
                                    for (int i = 0; i < 8; ++i)
                                        if ((mask[i * TC_MASK_WORDS + wd] >> (j & 31)) & 1u) x[i] += v;
                                }
                            }
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const long long at = at_s[g + i];
                        if (!whole)
                            P.part_o[at + t] = x[i];
                        else if (at >= 0)
                            static_cast<uint16_t*>(P.out)[at + t] = static_cast<uint16_t>(Ty::pack(x[i], 0.f));
                    }
                }
            }
            if (tid == 256 && w.u0 == 0 && !whole) P.desc[blockIdx.x] = make_int4(w.b, w.hr, w.parts(chunk), 0);
            tc_before();
            named_sync(3, 256);  // the groups' statistics are free
            if (dense) ++dseg;
            if (act) {
                if (lane == 0) sc_arrive(&q_empty[seg & 1]);
                ++seg;
            }
        }
    }
    if (failed) *err_s = 1;
    __syncwarp();
    tc_before();
    __syncthreads();
    if (warp == 17) {
        // the MMAs of a CTA that stopped early may still be running: free tensor memory after them
        if (!sc_wait(done, 0, P.timeout_ns)) *err_s = 1;
        __syncwarp();
        tc_after();
        tc_dealloc(tmem, 512);
        if (lane == 0 && *err_s && !P.whole) P.desc[blockIdx.x].w = 1;
    }
}

}  // namespace sv
