// rows_tc.cu -- attention of up to 128 query rows per work item over the paged latent cache, on
// the tensor cores' two-CTA form (tcgen05.mma.cta_group::2), fed by TMA.
//
// A work item (rows.h) is a few consecutive tokens of one sequence with all their heads: 128
// rows, 64 in each CTA of a two-CTA cluster. Per tile of 128 cached rows (two pages A and B of
// the item's visible pages):
//   S  = Q [128 x 576] . K^T [576 x 128]     one MMA chain, N = 128: CTA r stages page A or B
//   O += P [128 x 128] . V [128 x 512]       two MMAs per 16 tokens, N = 256: CTA r stages the
//                                            columns [256 r, 256 r + 256) of both pages
// The two-CTA form with M = 128 keeps 64 rows per CTA and lays the accumulator out over all 128
// TMEM lanes: lane l holds row l % 64, and lanes 64..127 the second half of the N columns. So S
// (128 columns) takes 64 TMEM columns and O (512) takes 256; the other 192 hold six of Q's nine
// column chunks (each row in lanes l and l + 64, as the A operand wants it), the last three
// lie in shared memory. The softmax of a row is done by two threads of its own CTA (one per
// page); nothing but barriers crosses the cluster. Each MMA runs at the full rate of the tensor
// pipe (measured back to back: 32 cycles at N = 128 with A in tensor or in shared memory, 64 at
// N = 256), so a tile costs it 36 * 32 + 16 * 64 = 2176 cycles.
//
// The same cache bytes are staged twice, as K chunks and as V chunks, the second time out of L2:
// one descriptor serves both CTAs, so a K chunk must hold the same columns at the same place in
// both and a V chunk the same tokens, and no place can be both. What bounds the kernel is the time
// a chunk's load takes against the bytes that shared memory can keep in flight: with all of
// Q in shared memory and room for one tile's K alone a tile took 2.8 us (two chunks of up to 300
// tokens on up to 16.5k rows at 128 heads), now 1.5, of which the MMAs are 1.1; the space won for K
// is why Q lies in tensor memory. 128 sequences of 128 heads over 33 tiles run at 5.2 TB/s.
//
// Online softmax in the exp2 domain with a lazily raised reference: it is raised only when a
// score exceeds it by more than 2^8, and then to that score, so that a row's largest weight is
// mostly 1. P is rounded to bf16 (half a step, 2^-8 of each weight; the row sum is taken of the
// weights before rounding), which leaves a weight of 1 as it is: a row that sees one cached row
// returns it, and the error of one that sees few is that of rounding the output (times 1.41 with
// whole numbers as references, 1.06 for two visible rows and 1.16 for eight with the maximum).
// Scores, sums and O are fp32.
//
// Every role walks the cluster's segments with counters that run on across them: the loads of
// the next segment start while the last one's rows are written.
//
// Roles per CTA: warp 0 loads K, 7 V (one lane each); in the leader CTA warp 1 issues S and
// warp 6 P . V (converged, one elected lane); warps 2-5 (TMEM lane = thread) softmax and output;
// the last four warps bring Q, and for an FP8 cache eight widen the codes. Every wait is bounded.
#include "common.cuh"
#include "fp8.cuh"
#include "kernels.h"
#include "rows.h"
#include "rows_shared.cuh"
#include "sm100.cuh"

namespace mla {

namespace {

using namespace sm100;

constexpr int CH = 64 * 128;  // one chunk: 64 rows (tokens, or query rows) x 64 bf16
constexpr int NCH = 9;        // 576 / 64
constexpr int KGC = 3;        // K is handed over in groups of 3 chunks, released as S goes
constexpr int KG = NCH / KGC;  // groups of a tile
constexpr int NQT = 6;         // Q chunks in tensor memory
constexpr int K_SLOT = KGC * CH;
// V is handed over in pages of 256 columns: 4 chunks
constexpr int VC = 4;
constexpr int V_SLOT = VC * CH;
constexpr int VS = 2;          // pages in flight (a tile has 2)
constexpr int C_SLOT = V_SLOT / 2;   // FP8: the codes of a V page
constexpr int KC_SLOT = K_SLOT / 2;  // and of a K group

// Shared memory. K groups in flight: 4 (5 or 3 with a third V page were slower on balance); for
// an FP8 cache 2, which leaves room to fetch codes before their places are free.
template <bool FP8> struct Layout {
    static constexpr int KS = FP8 ? 2 : 4;
    static constexpr int KCS = FP8 ? 2 : 0;  // groups of K codes in flight
    static constexpr int CS = FP8 ? 2 : 0;   // pages of V codes in flight
    static constexpr int Q_OFF = 0;         // Q chunks 6..8
    static constexpr int K_OFF = Q_OFF + (NCH - NQT) * CH;
    static constexpr int V_OFF = K_OFF + KS * K_SLOT;
    static constexpr int P_OFF = V_OFF + VS * V_SLOT;  // P: per page 64 rows x 64 tokens, bf16
    static constexpr int C_OFF = P_OFF + 2 * CH;
    static constexpr int KC_OFF = C_OFF + CS * C_SLOT;
    static constexpr int T_OFF = KC_OFF + KCS * KC_SLOT;  // Q rows on their way to tensor memory
    static constexpr int BAR_OFF = T_OFF + 2 * CH;
    static constexpr int NBAR = 40;
    static constexpr int MISC_OFF = BAR_OFF + NBAR * 8;
    static constexpr int EXP_OFF = MISC_OFF + 16;  // FP8: row exponents of K and V codes
    static constexpr int XM_OFF = EXP_OFF + (KCS + CS) * 64;  // exchanged between a row's halves
    static constexpr int ITEM_OFF = XM_OFF + 2 * 128 * 4;
    static constexpr int SMEM_TOTAL = ITEM_OFF + 32 + 1024;
    static_assert(SMEM_TOTAL <= 232448, "shared memory budget");
    static_assert(EXP_OFF % 16 == 0 && BAR_OFF % 8 == 0 && NCH % KGC == 0, "layout");
    static_assert(CS == 0 || CS == VS, "V's codes are counted by the slots of V");
    // FP8: warps 8-11 widen K, 12-15 V; Q by the last four
    static constexpr int NTHREADS = FP8 ? 512 : 384;
    // unrolling of the products' outer loops: none for FP8, where the instruction caches are the
    // limit (34.8 -> 33.8 us at 64 sequences of 9 tiles; bf16 would go from 372 to 422 us for two
    // chunks of 300 tokens on 16k rows)
    static constexpr int UG = FP8 ? 1 : KG;
    static constexpr int Q_WARP = NTHREADS / 32 - 4;
};

constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t TM_O = 0;    // O: two blocks of 128 columns
constexpr uint32_t TM_S = 256;  // S: 64 columns
constexpr uint32_t TM_Q = 320;  // Q chunks: 32 columns each, two bf16 per column
static_assert(TM_Q + 32 * NQT == TMEM_COLS, "tensor memory budget");
constexpr uint64_t WAIT_NS = 1000000000ull;
constexpr uint64_t DRAIN_NS = 200000000ull;
constexpr float TAU = 8.0f;

constexpr uint32_t IDESC_S = idesc_bf16(128, 128, false, false);
constexpr uint32_t IDESC_PV = idesc_bf16(128, 256, false, true);

// ---------------------------------------------------------------- two-CTA forms
__device__ __forceinline__ void tmem_alloc2(uint32_t dst_smem, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem),
                 "r"(ncols)
                 : "memory");
}
__device__ __forceinline__ void tmem_relinquish2() {
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc2(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
                 : "memory");
}
// executed by a converged warp, performed where `issue` is set
__device__ __forceinline__ void tc_mma2_if(bool issue, uint32_t d_tmem, uint64_t adesc,
                                           uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
        " @q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(static_cast<uint32_t>(issue))
        : "memory");
}
// the same with A in tensor memory
__device__ __forceinline__ void tc_mma2_ts_if(bool issue, uint32_t d_tmem, uint32_t a_tmem,
                                              uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
        " @q tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(static_cast<uint32_t>(issue))
        : "memory");
}
// arrives on the mbarrier at this offset in both CTAs when all prior MMAs are done
__device__ __forceinline__ void tc_commit2_if(bool issue, uint32_t bar) {
    asm volatile(
        "{\n .reg .pred q;\n setp.ne.b32 q, %2, 0;\n"
        " @q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
        "[%0], %1;\n}\n" ::"r"(bar),
        "h"(static_cast<uint16_t>(3)), "r"(static_cast<uint32_t>(issue))
        : "memory");
}
// Tiled load of chunks z, z + 1, .. (64 columns each) of 64 rows from y on into this CTA's shared
// memory, chunk after chunk. The bytes complete on this CTA's mbarrier, or (pair) on one of either
// CTA of the pair. One instruction brings a whole group: with one for each chunk the copies, not
// the memory, were the limit.
__device__ __forceinline__ void tma_chunks(uint32_t dst, const void *map, uint32_t bar, int y, int z,
                                           uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(0), "r"(y), "r"(z), "l"(policy)
        : "memory");
}
__device__ __forceinline__ void tma_chunks_pair(uint32_t dst, const void *map, uint32_t bar, int y,
                                                int z, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        ".L2::cache_hint [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(0), "r"(y), "r"(z), "l"(policy)
        : "memory");
}
// Arrive on an mbarrier of either CTA. What it announces is tensor memory (ordered by tcgen05
// fences) or shared memory that the tensor cores read (ordered by the proxy fence before it), so
// it carries no cluster-scope release: that form took about 900 cycles a tile, twice.
__device__ __forceinline__ void mbar_arrive_remote(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// a value that is the same in the whole warp, for the compiler to know it is
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); }
// descriptor of a 128-byte-swizzled operand at saddr, as its two halves, so that stepping through
// the operand is one addition (in units of 16 bytes, to the low half)
struct Desc {
    uint32_t lo, hi;
    __device__ __forceinline__ uint64_t at(uint32_t bytes) const {
        uint64_t d;
        asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo + (bytes >> 4)), "r"(hi));
        return d;
    }
};
__device__ __forceinline__ Desc desc_sw128(uint32_t saddr, uint32_t lbo) {
    const uint64_t d = sdesc_sw128(saddr, lbo, 1024);
    return {uniform(static_cast<uint32_t>(d)), uniform(static_cast<uint32_t>(d >> 32))};
}

// Bounded wait as mbar_wait, suspended by the hardware for longer at a time: with a dozen waiting
// warps the polls themselves took issue slots from the softmax (mixed batch, back to back on one set
// of inputs, 288 -> 274 us).
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int *abort) {
    if (mbar_poll(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    while (true) {
        uint32_t ok;
        asm volatile(
            "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n"
            " selp.u32 %0, 1, 0, p;\n}\n"
            : "=r"(ok)
            : "r"(bar), "r"(parity), "r"(100000u)  // ns
            : "memory");
        if (ok) return true;
        if (*abort) return false;
        if (globaltimer_ns() - t0 > WAIT_NS) {
            *abort = 1;
            return false;
        }
    }
}

// both, by a converged warp; the answers are usually there and cost a round trip each
__device__ __forceinline__ bool wait_both(uint32_t b0, uint32_t par0, uint32_t b1, uint32_t par1,
                                          volatile int *abort) {
    const bool r0 = mbar_poll(b0, par0), r1 = mbar_poll(b1, par1);
    bool ok = r0 && r1;
    if (!ok) ok = wait_bar(b0, par0, abort) && wait_bar(b1, par1, abort);
    return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity) {
    if (mbar_test(bar, parity)) return;
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_test(bar, parity))
        if (globaltimer_ns() - t0 > DRAIN_NS) return;
}
__device__ __forceinline__ void st_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                      uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
                 "r"(d)
                 : "memory");
}
__device__ __forceinline__ uint4 ld_v4(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// FP8: 16 codes of a row of a chunk to the row's place there: 64 bf16, 128-byte swizzled as TMA
// writes them; at0, at1: where the row's 16-byte pieces 2q and 2q + 1 lie.
//
// A code's exponent and mantissa, put at the low end of bf16's exponent and the top of its
// mantissa, make the bf16 number value * 2^-120, subnormal codes included, and one product with
// s2 = 2^(120 + e) the exact value. The NaN codes, which no quantised finite row holds, come out as
// 480. Four instructions for a pair of codes; what bounds the FP8 form are the instruction caches,
// with the widening beside the softmax and the products: its code is short, and loops stay rolled.
__device__ __forceinline__ void widen16(const uint4 &in, uint32_t s2, uint32_t at0, uint32_t at1) {
    const uint32_t w[4] = {in.x, in.y, in.z, in.w};
    uint32_t o[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        // codes 2k and 2k + 1 as 16-bit numbers with their signs repeated above them; then the
        // highest of those is the sign, and exponent and mantissa lie 4 bits further up
        uint32_t u;
        if (k & 1) asm("prmt.b32 %0, %1, 0, 0xB3A2;" : "=r"(u) : "r"(w[k >> 1]));
        else asm("prmt.b32 %0, %1, 0, 0x9180;" : "=r"(u) : "r"(w[k >> 1]));
        const uint32_t t = (u << 4) & 0x87F087F0u;
        asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(o[k]) : "r"(t), "r"(s2));
    }
    st_v4(at0, o[0], o[1], o[2], o[3]);
    st_v4(at1, o[4], o[5], o[6], o[7]);
}
// Where a row's exponent e is above 7 (rows of more than 2^15) 2^(120 + e) does not fit in bf16: s2 is
// 2^127 then, and this the rest. Out of line, being rare.
__device__ __noinline__ void widen_more(uint32_t to0, uint32_t to1, const volatile int8_t *ex) {
#pragma unroll 1
    for (int j = 0; j < 2; ++j) {
        const uint32_t m = bf16x2_pow2(max(ex[8 * j] - 7, 0));
#pragma unroll 1
        for (int k = 0; k < 2; ++k) {
            const uint32_t at = (k ? to1 : to0) + j * 1024;
            uint4 u = ld_v4(at);
            asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(u.x) : "r"(m));
            asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(u.y) : "r"(m));
            asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(u.z) : "r"(m));
            asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(u.w) : "r"(m));
            st_v4(at, u.x, u.y, u.z, u.w);
        }
    }
}
// 16 rows of a chunk by a warp, this lane's being r0 and r0 + 8: with factors from their exponents
// ex[0] and ex[8].
struct WidenRows {
    const volatile int8_t *ex;
    uint32_t s0, s1;
    bool wide;  // some row of the warp has an exponent above 7
    __device__ __forceinline__ explicit WidenRows(const volatile int8_t *e) : ex(e) {
        const int e0 = ex[0], e1 = ex[8];
        s0 = bf16x2_pow2(min(120 + max(e0, -126), 127));
        s1 = bf16x2_pow2(min(120 + max(e1, -126), 127));
        wide = __any_sync(0xffffffffu, max(e0, e1) > 7);
    }
    // from: the codes of row r0 (of 8 rows a load); to: its first piece's place (second: ^ 16)
    __device__ __forceinline__ void operator()(uint32_t from, uint32_t to) const {
        const uint4 a = ld_v4(from), b = ld_v4(from + 512);
        widen16(a, s0, to, to ^ 16);
        widen16(b, s1, to + 1024, (to ^ 16) + 1024);
        if (wide) widen_more(to, to ^ 16, ex);
    }
};

// The two warps of a pair meet at a CTA barrier; with a condition that holds for all, or for any,
// of their threads.
__device__ __forceinline__ void meet(int id) { asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory"); }
__device__ __forceinline__ bool meet_all(int id, bool v) {
    uint32_t all;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 q, %2, 0;\n bar.red.and.pred p, %1, 64, q;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(all)
        : "r"(id), "r"(static_cast<uint32_t>(v))
        : "memory");
    return all != 0;
}
__device__ __forceinline__ bool meet_any(int id, bool v) { return !meet_all(id, !v); }

// Whether one of the scores is a NaN or an infinity: 0 * x is 0 for every other x.
__device__ __forceinline__ bool not_finite(const uint32_t (&s)[64]) {
    uint64_t z[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 32; ++j)
        asm("{\n .reg .b64 x;\n mov.b64 x, {%1, %2};\n fma.rn.f32x2 %0, x, %3, %0;\n}\n"
            : "+l"(z[j & 3])
            : "r"(s[2 * j]), "r"(s[2 * j + 1]), "l"(0ull));
#pragma unroll
    for (int j = 2; j >= 1; j >>= 1)
#pragma unroll
        for (int k = 0; k < j; ++k) asm("add.rn.f32x2 %0, %0, %1;" : "+l"(z[k]) : "l"(z[k + j]));
    uint32_t a, b;
    asm("mov.b64 {%0, %1}, %2;" : "=r"(a), "=r"(b) : "l"(z[0]));
    return !(__uint_as_float(a) + __uint_as_float(b) == 0.f);
}
// whether one of two bf16 values is
__device__ __forceinline__ bool not_finite_bf16x2(uint32_t w) {
    return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u;
}

struct Segment {
    int b, tok0, ntok, pos0, t0, t1, part;  // part -1: the item's only segment
    VisiblePages v;
    const SharedPage *page;  // SHARED: of the item, from its first on
};

// Units of a ring so far: slot, and parity of the slot's round.
template <int N>
struct Ring {
    int slot = 0, round = 0;
    __device__ __forceinline__ void next() {
        if (++slot == N) slot = 0, round ^= 1;
    }
    __device__ __forceinline__ void back() {
        if (--slot < 0) slot = N - 1, round ^= 1;
    }
};

// SHARED: items are sequences that share a prefix, over the pages of rows_shared.cuh.
template <bool FP8, bool SHARED>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Layout<FP8>::NTHREADS, 1)
    rows_tc_kernel(const __grid_constant__ CUtensorMap map_k,
                   const __grid_constant__ CUtensorMap map_v,
                   const __grid_constant__ CUtensorMap map_ql,
                   const __grid_constant__ CUtensorMap map_qr, RowsParams p) {
    using LY = Layout<FP8>;
    constexpr int KS = LY::KS, KCS = LY::KCS, CS = LY::CS, Q_OFF = LY::Q_OFF, K_OFF = LY::K_OFF,
                  V_OFF = LY::V_OFF, P_OFF = LY::P_OFF, C_OFF = LY::C_OFF, KC_OFF = LY::KC_OFF,
                  T_OFF = LY::T_OFF, MISC_OFF = LY::MISC_OFF, EXP_OFF = LY::EXP_OFF,
                  XM_OFF = LY::XM_OFF, ITEM_OFF = LY::ITEM_OFF;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t sb = (raw + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (sb - raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_ctarank();
    const bool lead = rank == 0;

    // barriers: [L] lives in the leader, signalled from both CTAs; [B] in both, by the leader's
    // commits; [O] each CTA's own
    const uint32_t bar = sb + LY::BAR_OFF;
    auto k_full = [&](int g) { return bar + 8u * g; };             // [L] K slot in both CTAs
    auto k_empty = [&](int g) { return bar + 8u * (KS + g); };     // [B]
    auto kc_full = [&](int g) { return bar + 8u * (2 * KS + g); };  // [O] FP8: codes of a K group
    auto kc_empty = [&](int g) { return bar + 8u * (2 * KS + KCS + g); };  // [O] have been read
    const uint32_t rest = bar + 8u * (2 * KS + 2 * KCS);
    auto v_full = [&](int g) { return rest + 8u * g; };            // [O] V page in its slot
    auto v_empty = [&](int g) { return rest + 8u * (VS + g); };    // [B]
    auto vc_full = [&](int g) { return rest + 8u * (2 * VS + g); };  // [O] FP8: codes of a V page
    auto vc_empty = [&](int g) { return rest + 8u * (2 * VS + CS + g); };  // [O] have been read
    const uint32_t rest2 = rest + 8u * (2 * VS + 2 * CS);
    const uint32_t s_full = rest2;                                 // [B]
    const uint32_t s_free = rest2 + 8;                             // [L] 8 warps have read S
    const uint32_t q_full = rest2 + 16;                            // [L] 8 warps and TMA
    const uint32_t q_empty = rest2 + 24;                           // [B]
    // [L] P and V of page g are there, for page A also O as its reference wants it
    auto p_ready = [&](int g) { return rest2 + 32 + 8u * g; };
    auto pv_done = [&](int g) { return rest2 + 48 + 8u * g; };     // [B] P . V of page g is done
    const uint32_t o_free = rest2 + 64;                            // [L] 8 warps have read O
    static_assert(2 * (KS + KCS + VS + CS) + 9 <= LY::NBAR, "mbarrier count");
    auto at_lead = [&](uint32_t b) { return mapa(b, 0); };
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + MISC_OFF);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + MISC_OFF + 4);

    if (tid == 0) {
        for (int g = 0; g < KS; ++g) {
            // bf16: the leader's producer, with the bytes of both CTAs; FP8: four warps of each
            mbar_init(k_full(g), FP8 ? 8 : 1);
            mbar_init(k_empty(g), 1);
        }
        for (int g = 0; g < KCS; ++g) {
            mbar_init(kc_full(g), 1);
            mbar_init(kc_empty(g), 4);
        }
        for (int g = 0; g < VS; ++g) {
            mbar_init(v_full(g), FP8 ? 4 : 1);
            mbar_init(v_empty(g), 1);
        }
        for (int g = 0; g < CS; ++g) {
            mbar_init(vc_full(g), 1);
            mbar_init(vc_empty(g), 4);
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(p_ready(x), x == 0 ? 8 : 4);
            mbar_init(pv_done(x), 1);
        }
        mbar_init(s_full, 1);
        mbar_init(s_free, 8);
        mbar_init(q_full, 9);
        mbar_init(q_empty, 1);
        mbar_init(o_free, 8);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_map(&map_k);
        tma_prefetch_map(&map_v);
        tma_prefetch_map(&map_ql);
        tma_prefetch_map(&map_qr);
    }
    if (warp == 1) {
        tmem_alloc2(smem_u32(tmem_slot), TMEM_COLS);
        tmem_relinquish2();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers exist before anything is signalled
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    grid_dependency_wait();
    grid_launch_dependents();

    // ------------------------------------------------------------- this cluster's segments
    const int cl = blockIdx.x >> 1;
    const bool sched = SHARED || p.segs != nullptr;
    RowsSegment *own = reinterpret_cast<RowsSegment *>(smem + ITEM_OFF);  // fixed ranges: the one
    int2 list = make_int2(0, 0);
    if constexpr (SHARED) {
        // in the rings' memory, before anything is loaded there; the warps that bring Q go ahead as
        // soon as the segments are known (Q in its place is what the first scores wait for)
        static_assert(SHARED_SCRATCH <= T_OFF - K_OFF, "the rings' memory");
        SharedList work(p, smem + K_OFF);
        list = shared_list(p, work, cl, blockIdx.x == 0, own);
        fence_proxy_async_smem();
        if (warp < LY::Q_WARP) {
            shared_pages(p, work, list, cl, 32 * LY::Q_WARP);
            fence_proxy_async_smem();
            asm volatile("bar.sync 3, %0;" ::"r"(LY::NTHREADS) : "memory");
        } else {
            asm volatile("bar.arrive 3, %0;" ::"r"(LY::NTHREADS) : "memory");
        }
    }
    if (!sched) {
        if (warp == 0) {
            const int n = cl / p.num_splits, split = cl % p.num_splits;
            bool broken = false;
            const int4 it = p.q_starts ? find_item(p.q_starts, p.B, p.tokens, p.s_q, n, &broken)
                                       : make_int4(n, n * p.s_q, p.s_q, 0);
            if (lane == 0) {
                const int count = p.q_starts ? p.q_starts[it.x + 1] - p.q_starts[it.x] : p.s_q;
                const int L = min(max(p.seqlens[it.x], 0), p.max_seqlen);
                const int pos0 = L - count + it.w;
                const int t0 = split * p.tiles_per_split;
                const int end = visible_tiles(visible_pages(pos0, it.z, p.window, p.sinks));
                const int t1 = max(t0, min(t0 + p.tiles_per_split, end));
                *own = {it.x, it.y, it.z, pos0, t0, t1, p.num_splits > 1 ? cl : -1, 0};
                if (broken && blockIdx.x == 0) flag_error(p.err, MLA_ERR_OUT_OF_RANGE, 0);
            }
        }
        __syncthreads();
    }
    const int seg_begin = SHARED ? list.x : sched ? p.seg_range[2 * cl] : 0;
    const int seg_end = SHARED ? list.y : sched ? p.seg_range[2 * cl + 1] : own->ntok > 0;
    auto segment = [&](int i) {
        Segment s;
        const int4 *w =
            reinterpret_cast<const int4 *>(SHARED  ? i == seg_begin ? own : p.sh.segs + i
                                           : sched ? p.segs + i
                                                   : own);
        const int4 u = w[0], t = w[1];
        s.b = u.x, s.tok0 = u.y, s.ntok = u.z, s.pos0 = u.w;
        s.t0 = t.x, s.t1 = t.y, s.part = t.z;
        if constexpr (SHARED) s.page = p.sh.pages + 2 * (size_t)t.w;
        else s.v = visible_pages(s.pos0, s.ntok, p.window, p.sinks);
        return s;
    };
    // row of the page in the pool, or the first row past it (which TMA fills with zeros) for a
    // page that is not there or whose id is bad
    const int no_row = p.num_blocks * BLOCK;
    auto page_id = [&](const Segment &s, int v) {
        if constexpr (SHARED) return s.page[v].id;
        if (v >= s.v.count) return -2;
        return p.block_table[(size_t)s.b * p.max_blocks + (v < s.v.lead ? v : v + s.v.gap)];
    };
    auto in_pool = [&](int id) { return id >= 0 && id < p.num_blocks; };

    if (!sched && tid == 0 && rank == 0) {
        // the lengths, of sequences without tokens too
        for (int b = cl; b < p.B; b += gridDim.x >> 1) {
            const int L = p.seqlens[b];
            if (L < 0 || L > p.max_seqlen) flag_error(p.err, MLA_ERR_OUT_OF_RANGE, b);
        }
    }

    int tr = 0;  // tiles so far, over all segments
    if (warp == 0) {
        // ------------------------------------------------------------------ K producer
        if (lane == 0) {
            const uint64_t keep = l2_policy_evict_normal();  // read again as V
            Ring<FP8 ? KCS : KS> k;
            int groups = 0;
            bool ok = true;
            for (int i = seg_begin; ok && i < seg_end; ++i) {
                const Segment s = segment(i);
                int id = s.t0 < s.t1 ? page_id(s, 2 * s.t0 + rank) : 0;
                for (int t = s.t0; ok && t < s.t1; ++t) {
                    const bool there = in_pool(id);
                    if (!there && id != -2) flag_error(p.err, MLA_ERR_OUT_OF_RANGE, s.b);
                    const int y = there ? id * BLOCK : no_row;
                    const int now = id;
                    if (t + 1 < s.t1) id = page_id(s, 2 * (t + 1) + rank);
                    for (int g = 0; g < KG; ++g, ++groups, k.next()) {
                        // FP8: codes, ahead of their place
                        if (!(ok = wait_bar(FP8 ? kc_empty(k.slot) : k_empty(k.slot), k.round ^ 1,
                                            abort_flag)))
                            break;
                        if (FP8) {
                            const uint32_t full = kc_full(k.slot);
                            mbar_arrive_expect_tx(full, KC_SLOT + (there ? BLOCK : 0));
                            tma_chunks(sb + KC_OFF + k.slot * KC_SLOT, &map_k, full, y, g * KGC, keep);
                            if (there)
                                bulk_load(sb + EXP_OFF + 64 * k.slot, p.exps + (size_t)now * BLOCK,
                                          BLOCK, full);
                        } else {
                            if (lead) mbar_arrive_expect_tx(k_full(k.slot), 2 * K_SLOT);
                            tma_chunks_pair(sb + K_OFF + k.slot * K_SLOT, &map_k,
                                            at_lead(k_full(k.slot)), y, g * KGC, keep);
                        }
                    }
                }
            }
            // every load has been consumed, which is the leader's last signal for its slot (FP8: the
            // widening warps wait for that)
            for (int j = 0; !FP8 && j < KS && j < groups; ++j) {
                k.back();
                drain_wait(k_empty(k.slot), k.round);
            }
        }
    } else if (warp == 7) {
        // ------------------------------------------------------------------ V producer
        if (lane == 0) {
            const uint64_t last =
                p.stream_cache ? l2_policy_evict_first() : l2_policy_evict_normal();
            Ring<VS> v;
            int pages = 0;
            bool ok = true;
            for (int i = seg_begin; ok && i < seg_end; ++i) {
                const Segment s = segment(i);
                int id = s.t0 < s.t1 ? page_id(s, 2 * s.t0) : 0;
                for (int vp = 2 * s.t0; ok && vp < 2 * s.t1; ++vp, ++pages, v.next()) {
                    const bool there = in_pool(id);
                    const int now = id;
                    if (vp + 1 < 2 * s.t1) id = page_id(s, vp + 1);
                    const int y = there ? now * BLOCK : no_row;
                    if (FP8) {
                        // codes, ahead of their place
                        if (!(ok = wait_bar(vc_empty(v.slot), v.round ^ 1, abort_flag))) break;
                        const uint32_t full = vc_full(v.slot);
                        mbar_arrive_expect_tx(full, C_SLOT + (there ? BLOCK : 0));
                        tma_chunks(sb + C_OFF + v.slot * C_SLOT, &map_v, full, y, VC * rank, last);
                        if (there)
                            bulk_load(sb + EXP_OFF + 64 * (KCS + v.slot), p.exps + (size_t)now * BLOCK,
                                      BLOCK, full);
                    } else {
                        if (!(ok = wait_bar(v_empty(v.slot), v.round ^ 1, abort_flag))) break;
                        mbar_arrive_expect_tx(v_full(v.slot), V_SLOT);
                        tma_chunks(sb + V_OFF + v.slot * V_SLOT, &map_v, v_full(v.slot), y, VC * rank,
                                   last);
                    }
                }
            }
            for (int j = 0; !FP8 && j < VS && j < pages; ++j) {
                v.back();
                drain_wait(v_empty(v.slot), v.round);
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------------ S = Q . K^T
        if (lead) {
            const bool leader = elect_one();
            auto wait_all = [&](uint32_t b, uint32_t par) {
                return __all_sync(0xffffffffu, wait_bar(b, par, abort_flag));
            };
            Ring<KS> k;
            int qs = 0;
            bool ok = true;
            const uint32_t sd = uniform(tmem + TM_S), qt = uniform(tmem + TM_Q);
            const Desc qd = desc_sw128(sb + Q_OFF, 16);
            for (int i = seg_begin; ok && i < seg_end; ++i) {
                const Segment s = segment(i);
                if (s.t0 >= s.t1) continue;
                if (!(ok = wait_all(q_full, qs & 1))) break;
                for (int t = s.t0; ok && t < s.t1; ++t, ++tr) {
                    if (tr > 0 && !(ok = wait_all(s_free, (tr - 1) & 1))) break;
#pragma unroll(LY::UG)
                    for (int g = 0; g < KG; ++g) {
                        if (!(ok = wait_all(k_full(k.slot), k.round))) break;
                        tc_fence_after();
                        const Desc kd = desc_sw128(sb + K_OFF + k.slot * K_SLOT, 16);
                        static_assert(NQT % KGC == 0 && NCH - NQT == KGC, "Q of a group in one place");
                        if (g < NQT / KGC) {
                            const uint32_t qg = uniform(qt + 32 * KGC * g);
#pragma unroll
                            for (int c = 0; c < KGC; ++c)
#pragma unroll
                                for (int kk = 0; kk < 4; ++kk)
                                    tc_mma2_ts_if(leader, sd, qg + 32 * c + 8 * kk,
                                                  kd.at(c * CH + kk * 32), IDESC_S,
                                                  g > 0 || (c | kk) != 0);
                        } else {
#pragma unroll
                            for (int c = 0; c < KGC; ++c)
#pragma unroll
                                for (int kk = 0; kk < 4; ++kk)
                                    tc_mma2_if(leader, sd, qd.at(c * CH + kk * 32),
                                               kd.at(c * CH + kk * 32), IDESC_S, 1);
                        }
                        tc_commit2_if(leader, k_empty(k.slot));
                        k.next();
                        __syncwarp();
                    }
                    if (!ok) break;
                    tc_commit2_if(leader, s_full);
                    if (t + 1 == s.t1) tc_commit2_if(leader, q_empty);
                    __syncwarp();
                }
                ++qs;
            }
        }
        __syncwarp();
    } else if (warp == 6) {
        // ------------------------------------------------------------------ O += P . V
        if (lead) {
            const bool leader = elect_one();
            auto wait_all = [&](uint32_t b, uint32_t par) {
                return __all_sync(0xffffffffu, wait_bar(b, par, abort_flag));
            };
            const uint32_t od = uniform(tmem + TM_O);
            Ring<VS> v;
            int qs = 0;
            bool ok = true;
            for (int i = seg_begin; ok && i < seg_end; ++i) {
                const Segment s = segment(i);
                if (s.t0 >= s.t1) continue;
                for (int t = s.t0; ok && t < s.t1; ++t, ++tr) {
                    // the rows of the segment before have been read
                    if (t == s.t0 && qs > 0 && !(ok = wait_all(o_free, (qs - 1) & 1))) break;
#pragma unroll(LY::UG)
                    for (int g = 0; g < 2; ++g) {
                        if (!(ok = wait_all(p_ready(g), tr & 1))) break;
                        tc_fence_after();
                        const Desc pg = desc_sw128(sb + P_OFF + g * CH, 16);
                        const Desc vd = desc_sw128(sb + V_OFF + v.slot * V_SLOT, CH);
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
#pragma unroll
                            for (int n = 0; n < 2; ++n)
                                tc_mma2_if(leader, od + 128 * n, pg.at(kk * 32),
                                           vd.at(2 * n * CH + kk * 2048), IDESC_PV,
                                           t > s.t0 || g > 0 || kk > 0);
                        tc_commit2_if(leader, v_empty(v.slot));
                        v.next();
                        tc_commit2_if(leader, pv_done(g));
                        __syncwarp();
                    }
                }
                ++qs;
            }
        }
        __syncwarp();
    } else if (FP8 && warp >= 8 && warp < LY::Q_WARP) {
        // ------------------------------------------------------------ FP8: K's codes to bf16
        // Four warps, 16 rows each of every group (pairs that take the groups in turn, half the rows
        // each: 35.8 us where this takes 32.6, 64 sequences of 9 tiles).
        const int r0 = 16 * (warp & 3) + (lane >> 2);  // a load reads 8 rows: this lane lane / 4
        const uint32_t swz = r0 * 128 + (((2 * (lane & 3)) ^ (r0 & 7)) << 4);
        Ring<KCS> c;
        Ring<KS> k;
        int groups = 0;
        bool ok = true;
        for (int i = seg_begin; ok && i < seg_end; ++i) {
            const Segment s = segment(i);
            for (int g = KG * s.t0; g < KG * s.t1; ++g, ++groups, c.next(), k.next()) {
                if (!(ok = wait_both(kc_full(c.slot), c.round, k_empty(k.slot), k.round ^ 1,
                                     abort_flag)))
                    break;
                const uint32_t to = sb + K_OFF + k.slot * K_SLOT + swz;
                const uint32_t from = sb + KC_OFF + c.slot * KC_SLOT + 1024 * (warp & 3) + 16 * lane;
                const volatile int8_t *ex =
                    reinterpret_cast<const volatile int8_t *>(smem + EXP_OFF + 64 * c.slot) + r0;
                const WidenRows widen(ex);
#pragma unroll 1
                for (int d = 0; d < KGC; ++d) widen(from + d * (CH / 2), to + d * CH);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(kc_empty(c.slot));
                    mbar_arrive_remote(at_lead(k_full(k.slot)));
                }
            }
        }
        // the leader's last signals
        for (int j = 0; j < KS && j < groups; ++j) {
            k.back();
            drain_wait(k_empty(k.slot), k.round);
        }
        __syncwarp();
    } else if (warp >= LY::Q_WARP) {
        // --------------------------------------------------------- Q; FP8: V's codes to bf16
        // Q, this CTA's 64 rows of the item: chunks 0..5 go through registers into tensor memory
        // (row l % 64 in lane l), the last three by TMA into shared memory. Rows past the item's
        // are zeros there and other rows of q here: rows of the products do not mix, and these
        // are never written out.
        // FP8: 16 rows each of every page of V.
        const int quad = warp & 3;
        const uint32_t tq = tmem + (static_cast<uint32_t>(quad * 32) << 16) + TM_Q;
        const uint64_t pol = l2_policy_evict_normal();
        Ring<VS> v;
        int qs = 0, pages = 0;
        bool ok = true;
        auto wait_w = [&](uint32_t b, uint32_t par) {
            return __all_sync(0xffffffffu, wait_bar(b, par, abort_flag));
        };
        for (int i = seg_begin; ok && i < seg_end; ++i) {
            const Segment s = segment(i);
            {
                // a load reads 128 bytes of each of 4 rows, a whole chunk takes 8; the lanes get
                // their rows by way of shared memory (a lane loading its own row touches 32 lines
                // an instruction: the lookups alone took 6000 cycles a segment at 128 heads)
                const int row0 = 64 * static_cast<int>(rank) + 32 * (quad & 1);
                const int live = s.ntok * p.hq - row0;  // rows of this warp's 32
                const uint4 *src = reinterpret_cast<const uint4 *>(
                                       p.q_lat + ((size_t)s.tok0 * p.hq + row0) * D_C) +
                                   (lane >> 3) * (D_C / 8) + (lane & 7);
                constexpr int NF = FP8 ? 2 : 3;  // chunks in flight (as registers allow)
                uint4 qv[NF][8];
                auto load = [&](int c, uint4(&u)[8]) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        u[j] = 4 * j + (lane >> 3) < live ? src[8 * c + 4 * j * (D_C / 8)]
                                                          : make_uint4(0u, 0u, 0u, 0u);
                };
                // before anything that waits for the lengths
#pragma unroll
                for (int c = 0; c < NF; ++c) load(c, qv[c]);
                if constexpr (SHARED)  // the others' lines come meanwhile
                    if (lane < live)
#pragma unroll
                        for (int c = NF; c < NQT; ++c)
                            asm volatile("prefetch.global.L1 [%0];" ::"l"(
                                p.q_lat + ((size_t)s.tok0 * p.hq + row0 + lane) * D_C + 64 * c));
                if (s.t0 >= s.t1) continue;
                // every S of the segment before is done
                if (!(ok = wait_w(q_empty, (qs & 1) ^ 1))) break;
                tc_fence_after();
                if (warp == LY::Q_WARP && lane == 0) {
                    const uint32_t full = at_lead(q_full);
                    const int y = s.tok0 * p.hq + 64 * static_cast<int>(rank);
                    if (lead) mbar_arrive_expect_tx(q_full, 2 * (NCH - NQT) * CH);
                    tma_chunks_pair(sb + Q_OFF, &map_ql, full, y, NQT, pol);
                    tma_chunks_pair(sb + Q_OFF + (8 - NQT) * CH, &map_qr, full, y, 0, pol);
                }
                __syncwarp();
#pragma unroll
                for (int c = 0; c < NQT; ++c) {
                    const uint32_t stage = sb + T_OFF + 4096 * quad;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int row = 4 * j + (lane >> 3);
                        const uint4 u = qv[c % NF][j];
                        st_v4(stage + row * 128 + (((lane & 7) ^ (row & 7)) << 4), u.x, u.y, u.z,
                              u.w);
                    }
                    __syncwarp();
                    uint32_t w[32];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const uint4 u = ld_v4(stage + lane * 128 + ((j ^ (lane & 7)) << 4));
                        w[4 * j] = u.x, w[4 * j + 1] = u.y, w[4 * j + 2] = u.z, w[4 * j + 3] = u.w;
                    }
                    __syncwarp();
                    tmem_st32(tq + 32 * c, w);
                    if (c + NF < NQT) load(c + NF, qv[c % NF]);
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_remote(at_lead(q_full));
                ++qs;
            }
            if constexpr (FP8) {
                for (int vp = 2 * s.t0; vp < 2 * s.t1; ++vp, ++pages, v.next()) {
                    if (!(ok = wait_both(vc_full(v.slot), v.round, v_empty(v.slot), v.round ^ 1,
                                         abort_flag)))
                        break;
                    const int r0 = 16 * quad + (lane >> 2);
                    const uint32_t to = sb + V_OFF + v.slot * V_SLOT + r0 * 128 +
                                        (((2 * (lane & 3)) ^ (r0 & 7)) << 4);
                    const uint32_t from = sb + C_OFF + v.slot * C_SLOT + 1024 * quad + 16 * lane;
                    const volatile int8_t *ex =
                        reinterpret_cast<const volatile int8_t *>(smem + EXP_OFF +
                                                                  64 * (KCS + v.slot)) + r0;
                    const WidenRows widen(ex);
#pragma unroll 1
                    for (int c = 0; c < VC; ++c) widen(from + c * (CH / 2), to + c * CH);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(vc_empty(v.slot));
                        mbar_arrive(v_full(v.slot));
                    }
                }
            }
        }
        // the leader's last signals, on V's places (FP8; else V's producer waits for them) and on Q
        for (int j = 0; FP8 && j < VS && j < pages; ++j) {
            v.back();
            drain_wait(v_empty(v.slot), v.round);
        }
        if (qs > 0) drain_wait(q_empty, (qs - 1) & 1);
        __syncwarp();
    } else if (warp >= 2 && warp < 6) {
        // ------------------------------------------------------------- softmax / output
        const int quad = warp & 3;          // TMEM lanes 32 quad .. + 31
        const int tl = quad * 32 + lane;    // TMEM lane
        const int half = tl >> 6;           // page A or B of a tile; output columns 256 half ..
        const int r = tl & 63;              // row in this CTA
        const int row = 64 * static_cast<int>(rank) + r;  // row of the item
        const uint32_t ta = tmem + (static_cast<uint32_t>(quad * 32) << 16);
        volatile float *xm = reinterpret_cast<volatile float *>(smem + XM_OFF);  // row maxima
        volatile float *xl = xm + 128;                                            // row sums
        const uint32_t prow = sb + P_OFF + half * CH + (r >> 3) * 1024 + (r & 7) * 128;
        const int pair_id = 1 + (quad & 1);  // the two warps that share these 32 rows
        Ring<VS> v;
        bool ok = true;
        auto wait_w = [&](uint32_t b, uint32_t par) {
            return __all_sync(0xffffffffu, wait_bar(b, par, abort_flag));
        };
        // The CTA barriers of the two warps of a pair wait without a limit: both pass all of them,
        // also after a bounded wait of one has failed (the loops below go on without work then,
        // and nothing between two meetings waits for longer than its limit).
        auto arrive_lead = [&](uint32_t b) {
            __syncwarp();
            if (lane == 0) mbar_arrive_remote(at_lead(b));
        };
        for (int i = seg_begin; i < seg_end; ++i) {
            const Segment s = segment(i);
            const int rows = s.ntok * p.hq;
            const bool live = row < rows;
            int pos = live ? s.pos0 + row / p.hq : -1;  // last row this query sees
            // SHARED: the item's sequence that the row is of, and the last row that it sees of the
            // pages in common (those that its sequence fills)
            int seq = -1, pos_common = -1;
            if constexpr (SHARED) {
                pos = -1;
                if (live) {
                    seq = row / (p.s_q * p.hq);
                    const int L = min(max(p.seqlens[s.b + seq], 0), p.max_seqlen);
                    pos = L - p.s_q + (row / p.hq - seq * p.s_q);
                    pos_common = min(pos, min(s.pos0, L / BLOCK) * BLOCK - 1);
                }
            }
            // SHARED: of the next page position, owner and rows
            int4 next = make_int4(0, 0, 0, 0);
            if constexpr (SHARED)
                if (s.t0 < s.t1) next = *reinterpret_cast<const int4 *>(s.page + 2 * s.t0 + half);
            // rows that any token of the item sees: [0, sinks) and [see_lo, see_end)
            const int see_end = s.pos0 + s.ntok;
            const int first = max(s.pos0, 0);
            const int see_lo = p.window > 0 && first >= p.window ? first - p.window + 1 : 0;
            float m = -INFINITY, l = 0.f;
            int id_next = !SHARED && s.t0 < s.t1 ? page_id(s, 2 * s.t0 + half) : 0;
            for (int t = s.t0; t < s.t1; ++t, ++tr) {
                const int vp = 2 * t + half;
                const bool there = in_pool(id_next);  // a page with a bad id is masked
                if (!SHARED && t + 1 < s.t1) id_next = page_id(s, vp + 2);
                // (a page past the list is masked as a whole, and its position might not be an int)
                int base = 0;
                if constexpr (SHARED) base = next.y;
                else if (vp < s.v.count) base = (vp < s.v.lead ? vp : vp + s.v.gap) * BLOCK;
                const int owner = next.z & ~PAGE_APART, rows_there = next.w;
                const bool apart = SHARED && (next.z & PAGE_APART);
                if constexpr (SHARED)
                    if (t + 1 < s.t1) next = *reinterpret_cast<const int4 *>(s.page + vp + 2);
                uint32_t sr[64];
                float mx = -INFINITY;
                bool odd = false;
                if (ok) ok = wait_w(s_full, tr & 1);
                if (ok) {
                    tc_fence_after();
                    tmem_ld32(ta + TM_S, *reinterpret_cast<uint32_t(*)[32]>(&sr[0]));
                    tmem_ld32(ta + TM_S + 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[32]));
                    tmem_ld_wait();
                    tc_fence_before();
                    arrive_lead(s_free);

                    if constexpr (SHARED) {
                        // A page that not all of the item's tokens see in full, with a cached row that
                        // is not finite: nor is any query's score of it, so every warp knows. Those
                        // who see it get NaN, from an infinite score of either sign too, ..
                        odd = apart && __any_sync(0xffffffffu, not_finite(sr));
                        if (odd) {
#pragma unroll
                            for (int j = 0; j < 64; ++j)
                                if ((sr[j] & 0x7F800000u) == 0x7F800000u) sr[j] = 0x7FC00000u;
                        }
                    }
                    // of the page's 64 rows this query sees j < hi that are below snk or at
                    // least lo
                    int hi = 0, lo = 0, snk = 0;
                    if constexpr (SHARED) {
                        const int last = owner == 0 ? pos_common : owner == seq + 1 ? pos : -1;
                        hi = min(rows_there, max(0, last + 1 - base));
                    } else if (there) {
                        hi = min(BLOCK, max(0, pos + 1 - base));
                        if (p.window > 0) {
                            lo = pos >= p.window ? min(BLOCK, max(0, pos - p.window + 1 - base)) : 0;
                            snk = min(BLOCK, max(0, p.sinks - base));
                        }
                    }
                    if (!__all_sync(0xffffffffu, hi == BLOCK && (lo == 0 || snk == BLOCK))) {
#pragma unroll
                        for (int j = 0; j < 64; ++j)
                            if (!(j < hi && (j >= lo || j < snk))) sr[j] = 0xFF800000u;  // -inf
                    }
                    float a[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) a[j] = __uint_as_float(sr[j]);
#pragma unroll
                    for (int j = 8; j < 64; ++j) a[j & 7] = fmaxf(a[j & 7], __uint_as_float(sr[j]));
#pragma unroll
                    for (int w = 4; w >= 1; w >>= 1)
#pragma unroll
                        for (int j = 0; j < w; ++j) a[j] = fmaxf(a[j], a[j + w]);
                    mx = a[0] * p.scale_log2;  // scale > 0
                }
                // A reference is raised in few tiles but the first: the halves exchange their
                // maxima only when a row of theirs wants it.
                if (meet_any(pair_id, mx > m + TAU)) {
                    xm[tl] = mx;
                    meet(pair_id);
                    mx = fmaxf(mx, xm[tl ^ 64]);
                    const bool raise = mx > m + TAU;
                    const float m_new = raise ? mx : m;
                    const float alpha = raise ? fast_exp2(m - m_new) : 1.f;
                    if (ok && t > s.t0 && (ok = wait_w(pv_done(1), (tr - 1) & 1))) {
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < 8; ++c) {
                            uint32_t o[32];
                            tmem_ld32(ta + TM_O + 32 * c, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
                            tmem_st32(ta + TM_O + 32 * c, o);
                        }
                        tmem_st_wait();
                        tc_fence_before();
                    }
                    l *= alpha;
                    m = m_new;
                }
                if (!ok) continue;
                const float nm = m != -INFINITY ? -m : 0.f;
                float es = 0.f;
                uint32_t pk[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    const float p0 = fast_exp2(fmaf(__uint_as_float(sr[2 * j]), p.scale_log2, nm));
                    const float p1 = fast_exp2(fmaf(__uint_as_float(sr[2 * j + 1]), p.scale_log2, nm));
                    pk[j] = pack_bf16x2(p0, p1);
                    es += p0 + p1;
                }
                l += es;
                // P . V of this page of the tile before is done: its half of P may be written.
                // Page A's product covers all of O, so it also waits for page B's warps, whose
                // lanes hold half of it; they say so once page A's product of the tile before is
                // done (no arrival may run ahead into the phase of that tile).
                if (tr > 0 && !(ok = wait_w(pv_done(0), (tr - 1) & 1))) continue;
                if (half == 1) {
                    arrive_lead(p_ready(0));
                    if (tr > 0 && !(ok = wait_w(pv_done(1), (tr - 1) & 1))) continue;
                }
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    st_v4(prow + ((k ^ (r & 7)) << 4), pk[4 * k], pk[4 * k + 1], pk[4 * k + 2],
                          pk[4 * k + 3]);
                // this CTA's V chunks have landed; rows of them that no token of the item sees
                // may hold anything, and 0 * NaN would reach O: cleared (a page that is not
                // there was loaded as zeros)
                int e = min(BLOCK, max(0, see_end - base));
                const int a0 = min(BLOCK, max(0, see_lo - base));
                const int k0 = p.window > 0 ? min(BLOCK, max(0, p.sinks - base)) : 0;
                bool clear = vp < s.v.count && (e < BLOCK || (a0 > 0 && k0 < a0));
                if constexpr (SHARED) {
                    e = rows_there;
                    clear = e > 0 && e < BLOCK;
                }
                if (half == 1) v.next();
                if (!(ok = wait_w(v_full(v.slot), v.round))) continue;
                if (clear) {
                    // 64 rows x 4 chunks x 8 pieces over the half's 64 threads
                    for (int u = r; u < BLOCK * 32; u += 64) {
                        const int j = u >> 5;
                        if (j < e && (SHARED || j >= a0 || j < k0)) continue;
                        st_v4(sb + V_OFF + v.slot * V_SLOT + ((u >> 3) & 3) * CH + j * 128 +
                                  (u & 7) * 16,
                              0u, 0u, 0u, 0u);
                    }
                }
                if (odd) {
                    // .. and for the others, whose weights of it are 0, its values become zeros
#pragma unroll 1
                    for (int u = r; u < BLOCK * 32; u += 64) {
                        const uint32_t at = sb + V_OFF + v.slot * V_SLOT + ((u >> 3) & 3) * CH +
                                            (u >> 5) * 128 + (u & 7) * 16;
                        const uint4 w = ld_v4(at);
                        if (not_finite_bf16x2(w.x) || not_finite_bf16x2(w.y) ||
                            not_finite_bf16x2(w.z) || not_finite_bf16x2(w.w))
                            st_v4(at, 0u, 0u, 0u, 0u);
                    }
                }
                if (half == 0) v.next();
                v.next();
                fence_proxy_async_smem();
                tc_fence_before();
                arrive_lead(p_ready(half));
            }
            // ------------------------------------------------------------------- output
            const bool any = s.t0 < s.t1;
            if (any && ok) ok = wait_w(pv_done(1), (tr - 1) & 1);
            xl[tl] = l;  // the row's sum over both halves
            meet(pair_id);
            l += xl[tl ^ 64];
            const bool good = any && ok;
            const float inv = good && l > 0.f ? 1.f / l : 0.f;
            const size_t grow = (size_t)s.tok0 * p.hq + row;
            const size_t prw = (size_t)max(s.part, 0) * p.rows_per_item + row;
            if (good) tc_fence_after();
            if (good || (any ? false : live)) {
#pragma unroll 1
                for (int c = 0; c < 8; ++c) {
                    uint32_t o[32];
                    if (good) {
                        tmem_ld32(ta + TM_O + 32 * c, o);
                        tmem_ld_wait();
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j) o[j] = 0u;
                    }
                    if (!live) continue;
#pragma unroll
                    for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * inv);
                    if (s.part < 0) {
                        uint16_t *dst = p.out + grow * D_C + 256 * half + 32 * c;
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            uint32_t w[8];
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                w[j] = pack_bf16x2(__uint_as_float(o[16 * k + 2 * j]),
                                                   __uint_as_float(o[16 * k + 2 * j + 1]));
                            st_global_v8(dst + 16 * k, w[0], w[1], w[2], w[3], w[4], w[5], w[6], w[7]);
                        }
                    } else {
                        const uint64_t pol = l2_policy_evict_last();
                        // SHARED: 32 bytes of each of the CTA's 128 TMEM lanes side by side, whole
                        // lines for every store
                        float *dst = SHARED ? p.o_part + ((size_t)(2 * s.part + rank) * 32 + 4 * c) * 1024 + 8 * tl
                                            : p.o_part + prw * D_C + 256 * half + 32 * c;
                        constexpr int STEP = SHARED ? 1024 : 8;
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            st_global_v8_hint(dst + STEP * k, o[8 * k], o[8 * k + 1], o[8 * k + 2],
                                              o[8 * k + 3], o[8 * k + 4], o[8 * k + 5], o[8 * k + 6],
                                              o[8 * k + 7], pol);
                    }
                }
            }
            if (any) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_remote(at_lead(o_free));
            }
            if (half == 0 && live && (good || !any)) {
                // (SHARED: a NaN stays one, so that the merge does not take the part for an empty one)
                const bool some = any && (SHARED ? l != 0.f : l > 0.f);
                const float lse = some ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
                if (s.part < 0) p.lse[grow] = lse;
                else p.lse_part[prw] = lse;
            }
        }
    }

    __syncthreads();
    if (*abort_flag && tid == 0) {
        // gave up: every load in flight lands before the pair ends (of a barrier's two parities
        // one is the phase that is still open)
        flag_error(p.err, MLA_ERR_TIMEOUT, blockIdx.x);
        for (int par = 0; par < 2; ++par) {
            for (int g = 0; g < KS; ++g) drain_wait(k_full(g), par);
            for (int g = 0; g < KCS; ++g) drain_wait(kc_full(g), par);
            for (int g = 0; g < VS; ++g) drain_wait(v_full(g), par);
            for (int g = 0; g < CS; ++g) drain_wait(vc_full(g), par);
            drain_wait(q_full, par);
        }
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // nothing is signalled across the pair from here on
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc2(tmem, TMEM_COLS);
    }
}

// ------------------------------------------------------------------------- host side

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                  const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                  const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static const EncodeTiledFn fn = []() -> EncodeTiledFn {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000,
                                             cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return nullptr;
        return reinterpret_cast<EncodeTiledFn>(ptr);
    }();
    return fn;
}

// rows x cols seen as chunks of 64 columns, boxes of box_chunks chunks of 64 rows, laid out chunk
// after chunk: bf16 128-byte swizzled, or bytes as they are
bool encode_chunks(CUtensorMap *m, const void *base, uint64_t cols, uint64_t rows,
                   uint32_t box_chunks, bool bytes) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const uint64_t size = bytes ? 1 : 2;
    cuuint64_t dims[3] = {64, rows, cols / 64};
    cuuint64_t strides[2] = {cols * size, 64 * size};
    cuuint32_t box[3] = {64, 64, box_chunks};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, bytes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
              const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              bytes ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool FP8, bool SHARED>
cudaError_t launch_variant(const CUtensorMap &k, const CUtensorMap &v, const CUtensorMap &ql,
                           const CUtensorMap &qr,
                           const RowsParams &p, dim3 grid, cudaStream_t stream) {
    cudaError_t e = cudaFuncSetAttribute(rows_tc_kernel<FP8, SHARED>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         Layout<FP8>::SMEM_TOTAL);
    if (e != cudaSuccess) return e;
    return launch_pdl(rows_tc_kernel<FP8, SHARED>, grid, dim3(Layout<FP8>::NTHREADS),
                      Layout<FP8>::SMEM_TOTAL, stream, k, v, ql, qr, p);
}

}  // namespace

int rows_tc_cluster_slots() {
    static const int slots = []() {
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.gridDim = dim3(2 * 1024, 1, 1);
        cfg.blockDim = dim3(Layout<true>::NTHREADS, 1, 1);
        cfg.dynamicSmemBytes = Layout<true>::SMEM_TOTAL;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        if (cudaFuncSetAttribute(rows_tc_kernel<true, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 Layout<true>::SMEM_TOTAL) == cudaSuccess &&
            cudaOccupancyMaxActiveClusters(&n, rows_tc_kernel<true, false>, &cfg) == cudaSuccess && n > 0)
            return n;
        cudaGetLastError();
        return device_sm_count() / 2;
    }();
    return slots;
}

cudaError_t launch_rows_tc(const RowsParams &p, int clusters, cudaStream_t stream) {
    CUtensorMap k, v, ql, qr;
    const uint64_t rows = (uint64_t)p.tokens * p.hq, cached = (uint64_t)p.num_blocks * BLOCK;
    const bool fp8 = p.codes != nullptr;
    const void *cache = fp8 ? static_cast<const void *>(p.codes) : p.cache;
    if (!encode_chunks(&k, cache, D_QK, cached, KGC, fp8) ||
        !encode_chunks(&v, cache, D_QK, cached, VC, fp8) ||
        !encode_chunks(&ql, p.q_lat, D_C, rows, 8 - NQT, false) ||
        !encode_chunks(&qr, p.q_rope, D_ROPE, rows, 1, false))
        return cudaErrorInvalidValue;
    const dim3 grid(2 * clusters);
    if (p.sh.group_starts)
        return p.codes ? launch_variant<true, true>(k, v, ql, qr, p, grid, stream)
                       : launch_variant<false, true>(k, v, ql, qr, p, grid, stream);
    return p.codes ? launch_variant<true, false>(k, v, ql, qr, p, grid, stream)
                   : launch_variant<false, false>(k, v, ql, qr, p, grid, stream);
}

}  // namespace mla
