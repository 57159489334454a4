// kv_attention_tc.cu -- attention of many query rows over the paged 8-bit
// cache, on the 5th-generation tensor cores (tcgen05 + TMEM).
//
// The mathematics of kv_few_rows.cuh: weights 2^e_j with e_j = x_j +
// log2(vs_j) - M, M a reference of each row that moves only when some e_j
// passes 15.9, so that the value scales stay out of the products and the
// weights fit fp16.  The rows of a tile are the tokens of one sequence times
// the query heads of one kv head, tokens outermost.
//
// A CTA works on tiles of 256 rows as two halves of 128 (128 / group * group,
// whole tokens), over 128 keys a step.  Per step and half, S = Q K^T (128 x 128
// x D) and out += P V (128 x D x 128); TMEM holds S and out of both halves, and
// P as fp16 over the S it came from, the A operand of the second product.  When
// a tile's rows fit one half, both halves take the same rows, each every other
// step, and are joined at the end: else one half's softmax would have nothing
// to run beside.
//  * Warps 0-3 and 4-7: softmax of a half, a row a thread: no exchange among
//    threads, out is rescaled in TMEM by the same thread in the rare step that
//    moves M.  They write the output.
//  * Warps 8-11: codes to operands, K in the activations' type (exact: 8 bits
//    fit bf16's), V in fp16 like P.  Global loads into registers a step ahead,
//    conversion, 128-byte-swizzled stores: K is the K-major B operand of S, V
//    the MN-major B operand of out, the same bytes row by row.  The conversion
//    is paid once for 256 rows.
//  * Warp 12: issues the MMAs.  While one half's softmax runs the tensor cores
//    work on the other half's out += P V and next S.
//  * Warp 13: lists the CTA's tiles ahead of the others, and brings Q by TMA.
//
// The work is cut as in kv_few_rows.cuh: a line of all tiles' steps, each
// causal tile with just the steps that its rows see, in equal shares; CTAs
// that share a tile add their parts up through the workspace, in order.  Where
// whole tiles come close to that, the longest first, they are dealt out whole.
//
// Bound by the chain of a step, 2.4 to 2.5 us for two halves of rows: a softmax
// takes 1.05 to 1.2 us, and its wait for the next S 1.2 us, in which the other
// half's products and softmax go on; the tensor cores need 1.07 us of it
// (S takes its operands from shared memory, 64 cycles for 16 dims).  Where one
// half's worth of rows is all there is a step takes 2.15 us, set by the
// conversion warps.
// Measured: a prompt of 8192 tokens (32 heads on 8, 128 dims, int8), 33,280
// steps, 219 an SM: 549 us, 1000 TFLOP/s, 0.52 of the measured matrix rate,
// tensor pipe 42 % active; 1920 tokens 50 us.  P is fp16 and the sums are fp32,
// for the reasons that kv_few_rows.cuh gives.  Tried and slower: S in two 64-key pieces (more operand reads),
// conversion by 8 warps (the softmax then spills), 16-key units over 6 warps,
// raw codes by TMA through the 24 KB of shared memory that are left (too few
// bytes in flight), one stage of K and V with Q doubled.
#include <cuda.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "kv.cuh"

namespace w4a16 {
namespace {

constexpr int kHalfRows = 128, kTileRows = kManyTileRows, kKeys = 128;
constexpr int kMaxSeqs = 512;             // sequences of a launch
constexpr int kMaxEntries = 640;          // entries of one (SHARED): 512 sequences and their groups
constexpr int kFlagShift = 26;            // SHARED: an entry's flags above its first row, 2^24 at most
constexpr int kMaxPairs = 1216;           // (sequence, row tile) pairs of a launch
constexpr int kShortSteps = 2;            // tiles of up to so many steps stay in one CTA
constexpr int kCost = 3;                  // steps that a tile's start and end count for in the shares
constexpr int kSorted = 256;              // up to so many pairs may be dealt out whole, the longest first
constexpr int kSoftWarps = 8, kConvWarps = 4;
constexpr int kThreads = 32 * (kSoftWarps + kConvWarps + 2);   // and the MMA issuer, the planner
constexpr int kDrainTries = 1 << 16;      // looks at a barrier, up to 20 us each, before leaving all the same
constexpr int kRing = 4;                  // tiles that the planner is ahead of the slowest role
constexpr float kRefStart = -3.402823466e38f, kTop = 15.9f, kHead = 14.0f;

struct ManyParams {
    KvAttentionArgs a;
    KvCache c;
    KvBatch b;
    int row_limit;                        // sequences with up to so many rows a kv head are another kernel's
    int half_rows;                        // rows of a half in use: whole tokens, at most 128
    int before, after;                    // rows before the first sequence's, after the last one's are this launch's
    int pair_first;                       // this launch's pairs: [pair_first, pair_first + kMaxPairs)
    float *parts;                         // [grid][2] parts of a tile
    unsigned long long *tickets;          // [grid]
    unsigned long long tag;
    int hold;                             // test hook (kv_holds)
    int *status;
    KvShare share;                        // of a call with SHARED: what its sequences are (kv_attention_shared.cu)
};

struct ManyTile {
    int q0, n, first;                     // the sequence's rows, new tokens, position of the first
    int pair, seq, len, head, row0, rows;
    int steps, sink, block0;              // key blocks [0, sink) and from block0 on
    int lo, hi;                           // its rows see positions below `sinks` and lo..hi
    long long begin;                      // on the line
    long long pages;                      // where its page ids begin in the block table (SHARED)
    int flags;                            // of the entry (SHARED)
};

// A tile with this CTA's steps [s0, s1) of it; s1 == 0 ends the list.
struct PlannedTile {
    ManyTile t;
    int s0, s1;
};

template <int D>
struct ManySmem {
    static constexpr int kBlockBytes = kKeys * 128;               // 128 rows of 64 fp16
    static constexpr int kBlocks = D / 64;
    static constexpr int kOperand = kBlocks * kBlockBytes;
    static constexpr int kStages = 2;                             // of K and V
    static constexpr int kQ = 0;                                  // two halves
    static constexpr int kK = kQ + 2 * kOperand;
    static constexpr int kV = kK + kStages * kOperand;
    static constexpr int kPre = kV + kStages * kOperand;                // line position of each pair, of one kv head
    static constexpr int kSeq = kPre + (kMaxPairs + 1) * 8 + 8;   // int4 {q0, n, len, pairs before}
    static constexpr int kPairSeq = kSeq + kMaxEntries * 16;         // sequence of each pair
    static constexpr int kOrder = kPairSeq + kMaxPairs * 2;       // pairs by falling steps
    static constexpr int kScale = kOrder + kSorted * 2;        // [4][8] float4 {ks, log2 vs, 1 / vs, -}
    static constexpr int kExchange = kScale + 4 * 8 * 16;                // (M, l) of the second half's rows
    static constexpr int kPlan = kExchange + kHalfRows * 8;
    static constexpr int kBars = kPlan + kRing * (int)sizeof(PlannedTile);
    static constexpr int kMisc = kBars + (24 + 2 * kRing) * 8;
    static constexpr int kEnd = kMisc + 256 + 1024;               // 1024: slack to align the base
};

__device__ __forceinline__ float ex2(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t pack_bf162(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
// two fp32 numbers in a 64-bit register, and the arithmetic on such pairs
__device__ __forceinline__ uint64_t pair_of(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float &x, float &y) { asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// the largest of a value and two words of scores
__device__ __forceinline__ float max3(float a, uint32_t b, uint32_t c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(__uint_as_float(b)), "f"(__uint_as_float(c)));
    return r;
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}
// The load alone; its registers are good after tmem_ld_wait on them.
__device__ __forceinline__ void tmem_ld32_start(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                   "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                   "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                   "+r"(r[30]), "+r"(r[31])::"memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
// 32 bytes, as two 16-byte stores to one sector
__device__ __forceinline__ void st_v8(void *dst, const uint32_t *w) {
    *reinterpret_cast<uint4 *>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
    *(reinterpret_cast<uint4 *>(dst) + 1) = make_uint4(w[4], w[5], w[6], w[7]);
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// A step's MMAs, issued by one elected lane of a converged warp, so that
// descriptors and addresses stay in uniform registers: issued from a
// diverged lane, each MMA cost three times its 32 cycles of arithmetic.
// Descriptors are a low word (address, leading offset) and a constant high
// word; 16 of the contraction's elements further is a constant step.  One
// statement a step: the election and the predicates are made once.  Predicate
// p starts the sum or goes on with it, q (an instruction descriptor is never 0)
// goes on.
//
// S = Q K^T: 64 dims are four steps of 32 bytes in a 128-byte row; `far` is
// the step to the next 64 dims.
template <int BLOCKS>
__device__ __forceinline__ void mma_scores(uint32_t d, uint32_t alo, uint32_t blo, uint32_t hi, uint32_t idesc) {
    static_assert(BLOCKS == 1 || BLOCKS == 2, "64 or 128 dims");
    static_assert(kKeys * 128 / 16 == 1024, "the step to the next 64 dims, below");
    if (BLOCKS == 2) {
        asm volatile(
            "{\n\t.reg .pred e, p, q;\n\t.reg .b64 a, b;\n\t.reg .b32 x, y;\n\telect.sync _|e, 0xffffffff;\n\t"
            "setp.ne.b32 p, %5, 0;\n\tsetp.ne.b32 q, %4, 0;\n\t"
            "add.u32 x, %1, 0;\n\tadd.u32 y, %2, 0;\n\tmov.b64 a, {x, %3};\n\tmov.b64 b, {y, %3};\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t"
            "add.u32 x, %1, 2;\n\tadd.u32 y, %2, 2;\n\tmov.b64 a, {x, %3};\n\tmov.b64 b, {y, %3};\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, q;\n\t"
            "add.u32 x, %1, 4;\n\tadd.u32 y, %2, 4;\n\tmov.b64 a, {x, %3};\n\tmov.b64 b, {y, %3};\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, q;\n\t"
            "add.u32 x, %1, 6;\n\tadd.u32 y, %2, 6;\n\tmov.b64 a, {x, %3};\n\tmov.b64 b, {y, %3};\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, q;\n\t"
            "add.u32 x, %1, 1024;\n\tadd.u32 y, %2, 1024;\n\tmov.b64 a, {x, %3};\n\tmov.b64 b, {y, %3};\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, q;\n\t"
            "add.u32 x, %1, 1026;\n\tadd.u32 y, %2, 1026;\n\tmov.b64 a, {x, %3};\n\tmov.b64 b, {y, %3};\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, q;\n\t"
            "add.u32 x, %1, 1028;\n\tadd.u32 y, %2, 1028;\n\tmov.b64 a, {x, %3};\n\tmov.b64 b, {y, %3};\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, q;\n\t"
            "add.u32 x, %1, 1030;\n\tadd.u32 y, %2, 1030;\n\tmov.b64 a, {x, %3};\n\tmov.b64 b, {y, %3};\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, q;\n\t"
            "}" ::"r"(d), "r"(alo), "r"(blo), "r"(hi), "r"(idesc), "r"(0)
            : "memory");
    } else {
        asm volatile(
            "{\n\t.reg .pred e, p, q;\n\t.reg .b64 a, b;\n\t.reg .b32 x, y;\n\telect.sync _|e, 0xffffffff;\n\t"
            "setp.ne.b32 p, %5, 0;\n\tsetp.ne.b32 q, %4, 0;\n\t"
            "add.u32 x, %1, 0;\n\tadd.u32 y, %2, 0;\n\tmov.b64 a, {x, %3};\n\tmov.b64 b, {y, %3};\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t"
            "add.u32 x, %1, 2;\n\tadd.u32 y, %2, 2;\n\tmov.b64 a, {x, %3};\n\tmov.b64 b, {y, %3};\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, q;\n\t"
            "add.u32 x, %1, 4;\n\tadd.u32 y, %2, 4;\n\tmov.b64 a, {x, %3};\n\tmov.b64 b, {y, %3};\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, q;\n\t"
            "add.u32 x, %1, 6;\n\tadd.u32 y, %2, 6;\n\tmov.b64 a, {x, %3};\n\tmov.b64 b, {y, %3};\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, q;\n\t"
            "}" ::"r"(d), "r"(alo), "r"(blo), "r"(hi), "r"(idesc), "r"(0)
            : "memory");
    }
}
// out (+)= P V: P in TMEM, 8 columns a step; 16 keys of V are 2048 bytes.
__device__ __forceinline__ void mma_output(uint32_t d, uint32_t a, uint32_t blo, uint32_t hi, uint32_t idesc,
                                           uint32_t accumulate) {
    static_assert(kKeys == 128, "eight steps");
    asm volatile(
        "{\n\t.reg .pred e, p, q;\n\t.reg .b64 b;\n\t.reg .b32 x, y;\n\telect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %5, 0;\n\tsetp.ne.b32 q, %4, 0;\n\t"
        "add.u32 x, %1, 0;\n\tadd.u32 y, %2, 0;\n\tmov.b64 b, {y, %3};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %4, p;\n\t"
        "add.u32 x, %1, 8;\n\tadd.u32 y, %2, 128;\n\tmov.b64 b, {y, %3};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %4, q;\n\t"
        "add.u32 x, %1, 16;\n\tadd.u32 y, %2, 256;\n\tmov.b64 b, {y, %3};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %4, q;\n\t"
        "add.u32 x, %1, 24;\n\tadd.u32 y, %2, 384;\n\tmov.b64 b, {y, %3};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %4, q;\n\t"
        "add.u32 x, %1, 32;\n\tadd.u32 y, %2, 512;\n\tmov.b64 b, {y, %3};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %4, q;\n\t"
        "add.u32 x, %1, 40;\n\tadd.u32 y, %2, 640;\n\tmov.b64 b, {y, %3};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %4, q;\n\t"
        "add.u32 x, %1, 48;\n\tadd.u32 y, %2, 768;\n\tmov.b64 b, {y, %3};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %4, q;\n\t"
        "add.u32 x, %1, 56;\n\tadd.u32 y, %2, 896;\n\tmov.b64 b, {y, %3};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %4, q;\n\t"
        "}" ::"r"(d), "r"(a), "r"(blo), "r"(hi), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void commit_elected(uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
        : "memory");
}

// A V tile as B: rows are keys (the contraction), 64 dims a 128-byte row,
// 128-byte swizzle, the next 64 dims a block further.  MN-major: the leading
// offset goes from 64 dims to the next, the stride offset from 8 keys to the
// next.
__device__ __forceinline__ uint64_t desc_mn_sw128(uint32_t saddr, uint32_t block_bytes) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
    d |= (uint64_t)(block_bytes >> 4) << 16;
    d |= (uint64_t)(1024 >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}

// Codes of a word as pairs (0, 1) and (2, 3) of fp16 (see kv_few_rows.cuh) or
// bf16, exactly.  int8 as bf16: 0x4300 with the low seven bits is 128 + those,
// 0x4300 with the sign bit is 128 or 256; their difference is the code.
template <int KT, bool BF16>
__device__ __forceinline__ void codes_to_act(uint32_t w, uint32_t &lo, uint32_t &hi) {
    if constexpr (KT == kKvInt8 && BF16) {
        const uint32_t low = w & 0x7f7f7f7fu, sign = w & 0x80808080u;
        const uint32_t a = __byte_perm(low, 0x43434343u, 0x4140), b = __byte_perm(low, 0x43434343u, 0x4342);
        const uint32_t c = __byte_perm(sign, 0x43434343u, 0x4140), d = __byte_perm(sign, 0x43434343u, 0x4342);
        const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&a), *reinterpret_cast<const __nv_bfloat162 *>(&c));
        const __nv_bfloat162 s = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&b), *reinterpret_cast<const __nv_bfloat162 *>(&d));
        lo = *reinterpret_cast<const uint32_t *>(&r), hi = *reinterpret_cast<const uint32_t *>(&s);
    } else if constexpr (KT == kKvInt8) {
        w ^= 0x80808080u;
        const uint32_t bias = 0x64806480u;
        const uint32_t x = __byte_perm(w, 0x64646464u, 0x4140), y = __byte_perm(w, 0x64646464u, 0x4342);
        const __half2 b = *reinterpret_cast<const __half2 *>(&bias);
        const __half2 r = __hsub2(*reinterpret_cast<const __half2 *>(&x), b);
        const __half2 s = __hsub2(*reinterpret_cast<const __half2 *>(&y), b);
        lo = *reinterpret_cast<const uint32_t *>(&r), hi = *reinterpret_cast<const uint32_t *>(&s);
    } else {
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t"
            "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
            : "=r"(lo), "=r"(hi)
            : "r"(w));
        if constexpr (BF16) {
            const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&lo));
            const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
            lo = pack_bf162(a.x, a.y), hi = pack_bf162(b.x, b.y);
        }
    }
}

// A lane's codes, 16-byte piece `piece` of rows row, row + ROWS, .., into an
// operand tile: 128-byte rows of 64 elements, 16-byte chunks at c ^ (row % 8).
template <int KT, int D, bool BF16>
__device__ __forceinline__ void convert_codes(const uint4 (&raw)[D == 128 ? 8 : 4], uint8_t *tile, int row, int piece) {
    constexpr int ROWS = D == 128 ? 4 : 8;
#pragma unroll
    for (int i = 0; i < (D == 128 ? 8 : 4); ++i, row += ROWS) {
        uint32_t h[8];
        codes_to_act<KT, BF16>(raw[i].x, h[0], h[1]);
        codes_to_act<KT, BF16>(raw[i].y, h[2], h[3]);
        codes_to_act<KT, BF16>(raw[i].z, h[4], h[5]);
        codes_to_act<KT, BF16>(raw[i].w, h[6], h[7]);
        uint8_t *dst = tile + (piece >> 2) * (kKeys * 128) + row * 128;
        const int c = 2 * piece & 7;
        *reinterpret_cast<uint4 *>(dst + ((c ^ (row & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
        *reinterpret_cast<uint4 *>(dst + (((c + 1) ^ (row & 7)) << 4)) = make_uint4(h[4], h[5], h[6], h[7]);
    }
}

template <bool SHARED, int KT, int D>
__global__ void __launch_bounds__(kThreads, 1) 
    many_rows_kernel(const __grid_constant__ CUtensorMap tm_q, const ManyParams p) {
    using L = ManySmem<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int Hk = p.c.n_kv_heads, group = p.a.n_heads / Hk, B = p.b.n_seqs, half_rows = p.half_rows;
    long long *pre = reinterpret_cast<long long *>(smem + L::kPre);
    int4 *seqs = reinterpret_cast<int4 *>(smem + L::kSeq);
    uint16_t *pair_seq = reinterpret_cast<uint16_t *>(smem + L::kPairSeq);
    float4 *scales = reinterpret_cast<float4 *>(smem + L::kScale);
    const uint32_t bars = smem_u32(smem + L::kBars);
    int *misc = reinterpret_cast<int *>(smem + L::kMisc);
    long long *s_cut = reinterpret_cast<long long *>(misc + 8);    // [2]
    long long *s_scan = s_cut + 2;                                 // [kThreads / 32]
    volatile int *abort_flag = misc;
    // barriers: halves' S ready, P ready, out ready, Q ready; stages of K and V full and empty
    auto s_full = [&](int i) { return bars + 8u * i; };
    auto p_ready = [&](int i) { return bars + 8u * (2 + i); };
    auto o_full = [&](int i) { return bars + 8u * (4 + i); };
    auto q_full = [&](int i) { return bars + 8u * (6 + i); };
    auto q_empty = [&](int i) { return bars + 8u * (22 + 2 * kRing + i); };
    auto k_full = [&](int i) { return bars + 8u * (8 + i); };
    auto k_empty = [&](int i) { return bars + 8u * (10 + i); };
    auto v_full = [&](int i) { return bars + 8u * (12 + i); };
    auto v_empty = [&](int i) { return bars + 8u * (14 + i); };
    const uint32_t drain = bars + 8u * 16;
    auto plan_full = [&](int i) { return bars + 8u * (18 + i); };
    auto plan_empty = [&](int i) { return bars + 8u * (18 + kRing + i); };
    const uint32_t part_told = bars + 8u * (18 + 2 * kRing), part_read = part_told + 8u;
    auto meet_bar = [&](int i) { return part_told + 8u * (2 + i); };
    PlannedTile *plan = reinterpret_cast<PlannedTile *>(smem + L::kPlan);

    if (tid == 0) {
        tma_prefetch_desc(&tm_q);
        for (int i = 0; i < 2; ++i) {
            mbar_init(s_full(i), 1);
            mbar_init(p_ready(i), kHalfRows);
            mbar_init(o_full(i), 1);
            mbar_init(q_full(i), 1);
            mbar_init(q_empty(i), 1);
            mbar_init(k_full(i), kConvWarps);
            mbar_init(k_empty(i), 1);
            mbar_init(v_full(i), kConvWarps);
            mbar_init(v_empty(i), 1);
        }
        mbar_init(drain, 1);
        mbar_init(part_told, kHalfRows);
        mbar_init(part_read, kHalfRows);
        mbar_init(meet_bar(0), kHalfRows);
        mbar_init(meet_bar(1), kTileRows);
        for (int i = 0; i < kRing; ++i) {
            mbar_init(plan_full(i), 1);
            mbar_init(plan_empty(i), kSoftWarps + kConvWarps + 1);
        }
        fence_mbar_init();
        misc[0] = misc[3] = 0;                                     // misc[3]: tickets taken, 1 the first tile's, 2 the last's
    }
    grid_dependency_wait();

    // the position tok tokens after `first`: all the same where every row sees all keys
    auto position = [](int flags, int first, int tok) { return flags & kKvOthers ? first + tok : first; };
    auto tile_of = [&](const int4 s, int b, int r) {
        ManyTile t;
        t.seq = b;
        t.flags = SHARED ? s.x >> kFlagShift : kKvOthers;
        t.q0 = SHARED ? s.x & (1 << kFlagShift) - 1 : s.x, t.n = s.y, t.len = s.z;
        t.first = t.flags & kKvOthers ? s.z - s.y : s.z - 1;
        t.row0 = r * 2 * half_rows;
        t.rows = min(2 * half_rows, s.y * group - t.row0);
        const int lo_pos = position(t.flags, t.first, t.row0 / group);
        const int hi_pos = position(t.flags, t.first, (t.row0 + t.rows - 1) / group);
        const int lo = p.a.window > 0 ? max(0, lo_pos + 1 - p.a.window) : 0;
        t.lo = lo, t.hi = hi_pos;
        t.block0 = lo / kKeys;
        t.sink = min((min(p.a.sinks, lo) + kKeys - 1) / kKeys, t.block0);
        t.steps = max(t.sink + (max(hi_pos + 1, 0) + kKeys - 1) / kKeys - t.block0, 1);
        t.pair = t.head = 0;
        t.begin = t.pages = 0;
        return t;
    };
    // Sum over the threads before this one, and of all; every thread calls.
    auto scan = [&](long long v, long long &all) {
        long long inc = v;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const long long x = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d) inc += x;
        }
        __syncthreads();
        if (lane == 31) s_scan[warp] = inc;
        __syncthreads();
        long long ahead = 0;
        all = 0;
        for (int w = 0; w < kThreads / 32; ++w) {
            const long long x = s_scan[w];
            ahead += w < warp ? x : 0;
            all += x;
        }
        return ahead + inc - v;
    };

    // ---- the line: pairs (sequence, row tile), then the steps of each, for one kv head
    int pairs = 0;
    for (int base = 0; base < B; base += kThreads) {
        const int i = base + tid;
        int4 s = make_int4(0, 0, 0, 0);
        int mine = 0;
        if (i < B) {
            KvSeq q;
            int flags = 0;                                         // above the bits of a row
            if constexpr (SHARED) {
                const KvEntry e = kv_entry(p.share, i);
                q = KvSeq{e.q0, (e.flags & kKvBig) && kv_division(p.share, 0) ? e.n : 0, e.len};
                flags = e.flags << kFlagShift;
            } else {
                q = kv_sequence(p.b, p.c.page_shift, i, p.status);
            }
            const int rows = q.n * group;
            mine = rows <= p.row_limit ? 0 : (rows + 2 * half_rows - 1) / (2 * half_rows);
            s = make_int4(q.q0 | flags, q.n, q.len, 0);
        }
        long long all;
        s.w = (int)scan(mine, all) + pairs - p.pair_first;         // within this launch's range
        if (i < B) seqs[i] = s;
        pairs += (int)all;
    }
    pairs = min(pairs - p.pair_first, kMaxPairs);
    __syncthreads();
    if (p.before | p.after)
        kv_empty_rows(p.a, p.b, D, p.before ? seqs[0].x : 0, p.after ? seqs[B - 1].x + seqs[B - 1].y : p.b.n_tokens);
    if (pairs <= 0) return;
    long long total = 0;
    for (int base = 0; base < pairs; base += kThreads) {
        const int i = base + tid;
        long long v = 0;
        if (i < pairs) {
            int lo = 0, hi = B - 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (seqs[mid].w <= i) lo = mid;
                else hi = mid - 1;
            }
            pair_seq[i] = (uint16_t)lo;
            v = tile_of(seqs[lo], lo, i - seqs[lo].w).steps + kCost;
        }
        long long all;
        const long long at = scan(v, all) + total;
        if (i < pairs) pre[i] = at;
        total += all;
    }
    if (tid == 0) pre[pairs] = total;
    total *= Hk;
    __syncthreads();

    // Whole tiles or equal shares?  With few tiles the longest first, dealt out to and fro, can come close to
    // equal shares without the parts that shared tiles leave; each thread adds up one CTA's hand.
    uint16_t *order = reinterpret_cast<uint16_t *>(smem + L::kOrder);
    const int grid = SHARED ? kv_division(p.share, 1) : gridDim.x;
    if (SHARED && blockIdx.x >= grid) return;
    auto dealt = [&](int cta, int round) { return round * grid + (round & 1 ? grid - 1 - cta : cta); };
    bool deal = false;
    if (pairs <= kSorted) {
        for (int i = tid; i < pairs; i += kThreads) {
            const long long mine = pre[i + 1] - pre[i];
            int rank = 0;
            for (int j = 0; j < pairs; ++j) {
                const long long x = pre[j + 1] - pre[j];
                rank += x > mine || (x == mine && j < i);
            }
            order[rank] = (uint16_t)i;
        }
        __syncthreads();
        long long most = 0;
        for (int cta = tid; cta < grid; cta += kThreads) {
            long long hand = 0;
            for (int round = 0; round * grid < pairs * Hk; ++round) {
                const int i = dealt(cta, round);
                if (i < pairs * Hk) hand += pre[order[i / Hk] + 1] - pre[order[i / Hk]];
            }
            most = max(most, hand);
        }
        for (int d = 16; d > 0; d >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, d));
        if (lane == 0) s_scan[warp] = most;
        __syncthreads();
        for (int w = 0; w < kThreads / 32; ++w) most = max(most, s_scan[w]);
        // Parts cost a CTA about 8 steps, and an eighth of its time: prompts of 300 / 1920 / 8192 tokens dealt whole
        // take 18 / 50 / 549 us, in shares 23 / 68 / 578; five tokens each over 24 contexts, where a whole tile is
        // most of a CTA's share, take 76 us dealt and 51 in shares.
        // Left for the join parts cost 2 or so: 16 groups of 100 to 1920 shared keys 97 us at 8 steps, 94 at 2.
        deal = SHARED && p.share.defer ? most <= total / grid + 2 + total / grid / 16 : most <= total / grid + 8 + total / grid / 8;
    }

    auto tile_at = [&](int pair, int head) {
        const int b = pair_seq[pair];
        const int4 s = seqs[b];
        ManyTile t = tile_of(s, b, pair - s.w);
        t.pair = pair, t.head = head;
        t.begin = pre[pair] * Hk + (long long)head * (t.steps + kCost);
        if (SHARED) t.pages = kv_entry_pages(p.share, b);
        return t;
    };
    auto find_pair = [&](long long at) {                           // the pair of a position of the line
        int lo = 0, hi = pairs - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (pre[mid] * Hk <= at) lo = mid;
            else hi = mid - 1;
        }
        return lo;
    };
    const long long ctas = min((long long)grid, (total + kCost) / (1 + kCost));
    if (deal ? (int)blockIdx.x >= pairs * Hk : blockIdx.x >= ctas) return;
    if (tid == 0) misc[4] = deal, misc[5] = pairs;
    if (tid < 2) {
        long long at = ((long long)blockIdx.x + tid) * total / ctas;
        if (at > 0 && at < total) {
            const int pair = find_pair(at);
            const long long each = pre[pair + 1] - pre[pair], rem = at - pre[pair] * Hk;
            if (each <= kShortSteps + kCost) at -= rem % each;
        }
        s_cut[tid] = at;
    }
    if (warp == kSoftWarps + kConvWarps) {
        tmem_alloc(smem_u32(misc + 1), 512u);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // The next kernel may start only now: one that takes TMEM before it waits for this grid must not have it first.
    grid_dependents_launch();
    const long long c0 = s_cut[0], c1 = s_cut[1];
    const uint32_t tmem = static_cast<uint32_t>(misc[1]);
    // the tile at c0, and the walk from there
    int pair = 0, head = 0;
    if (!deal && c0 < c1) {
        pair = find_pair(c0);
        head = (int)((c0 - pre[pair] * Hk) / (pre[pair + 1] - pre[pair]));
    }
    // Every wait is a whole warp's, and so is its giving up: what follows is full of warp-wide instructions.
    // In the MMA warp the vote is left until a step's end, off its chain: a step issued on what is not there touches
    // nothing but this CTA's operands and tensor memory.  A prompt of 8192 tokens takes 549 us so, 560 with a vote at each
    // of its waits; at a step's end in the conversion warps, with loads on their way, it costs more, 570.
    auto look = [&](uint32_t bar, int phase) { return mbar_wait_bounded(bar, phase, p.status, abort_flag); };
    auto all = [](bool ok) { return __all_sync(0xffffffffu, ok) != 0; };
    auto wait = [&](uint32_t bar, int phase) { return all(look(bar, phase)); };
    // The list of this CTA's tiles, written by the planner ahead of the other roles.  open_tile waits for
    // the idx-th (null: the end, or a wait that ran out), close_tile gives its place back.
    auto open_tile = [&](int idx) -> const PlannedTile * {
        if (!wait(plan_full(idx % kRing), (idx / kRing) & 1)) return nullptr;
        const PlannedTile *t = plan + idx % kRing;
        return t->s1 > 0 ? t : nullptr;
    };
    auto close_tile = [&](int idx) {
        __syncwarp();
        if (lane == 0) mbar_arrive(plan_empty(idx % kRing));
    };
    // A tile of up to a half's rows has both halves work on the same rows, each on every other step.
    auto same_rows = [&](const ManyTile &t) { return t.rows <= half_rows; };
    auto half_runs = [&](const PlannedTile &t, int half) { return same_rows(t.t) ? t.s1 - t.s0 > half : true; };
    auto block_of = [](const ManyTile &t, int st) { return st < t.sink ? st : t.block0 + st - t.sink; };

    // The CTAs that share a tile: the last whose share begins by its first step, and by its last.
    auto first_cta = [](const ManyTile &t, long long ctas, long long total) {
        return (int)(((t.begin + kCost + 1) * ctas + total - 1) / total - 1);
    };
    auto last_cta = [](const ManyTile &t, long long ctas, long long total) {
        return (int)(((t.begin + kCost + t.steps) * ctas + total - 1) / total - 1);
    };
    // This CTA's ticket of a shared tile, from one thread; true for the last to come.
    auto ticket = [&](int from, int to) {
        unsigned long long *tk = p.tickets + from, old = __ldcg(tk), seen, put;
        do {
            seen = old;
            const unsigned long long n = (seen >> 16) == p.tag ? (seen & 0xffff) + 1 : 1;
            put = n == (unsigned long long)(to - from + 1) ? 0 : p.tag << 16 | n;
            old = atomicCAS(tk, seen, put);
        } while (old != seen);
        return put == 0;
    };

    if (warp < kSoftWarps) {
        // ------------------------------------------------------------ softmax, Q, output
        const int half = warp >> 2, r = tid & 127;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t t_s = tmem + lanes + half * 128, t_o = tmem + lanes + 256 + half * D;
        int s_phase = 0, o_phase = 0, other_phase = 0, join_phase = 0, meet_phase[2] = {0, 0};
        float2 *exchange = reinterpret_cast<float2 *>(smem + L::kExchange);
        const int r_tok = r / group, r_head = r - r_tok * group;   // the row within its half: token and head
        const float my_fac = fabsf(p.a.scale) * 1.4426950408889634f;
        auto store = [&](long long at, int d0, const float (&v)[32], float inv) {
            uint16_t *dst = static_cast<uint16_t *>(p.a.out) + at * D + d0;
            uint32_t w[16];
#pragma unroll
            for (int j = 0; j < 16; ++j)
                w[j] = p.a.dtype == 0 ? pack_half2(v[2 * j] * inv, v[2 * j + 1] * inv)
                                      : pack_bf162(v[2 * j] * inv, v[2 * j + 1] * inv);
            // whole 32-byte sectors
#pragma unroll
            for (int j = 0; j < 16; j += 8) st_v8(dst + 2 * j, &w[j]);
        };
        int counter = 0;                                           // steps so far: the scales' ring position
        bool ok = true;
        for (int idx = 0; ok; ++idx) {
            const PlannedTile *next = open_tile(idx);
            if (!next) break;
            const ManyTile &t = next->t;                           // in shared memory
            const int s0 = next->s0, s1 = next->s1;
            const bool runs = half_runs(*next, half), twice = same_rows(t);
            const int base_row = twice ? 0 : half * half_rows;
            const int sink_blocks = t.sink, block0 = t.block0 - t.sink;
            const bool whole = s0 == 0 && s1 == t.steps, opens = s0 == 0;
            const bool exists = r < half_rows && base_row + r < t.rows;
            const int tok0 = (t.row0 + base_row) / group;          // the half's first token
            const int flags = SHARED ? t.flags : kKvOthers;
            const int min_pos = position(flags, t.first, tok0), pos = exists ? position(flags, min_pos, r_tok) : -1;
            const int max_pos = position(flags, t.first, (t.row0 + min(base_row + half_rows, t.rows) - 1) / group);
            float ref = kRefStart, sum = 0.0f;
            const int first_st = twice ? s0 + half : s0;
            for (int st = first_st; st < s1 && runs; st += twice ? 2 : 1) {
                const int pos0 = (st < sink_blocks ? st : block0 + st) * kKeys;
                const float4 *sc = scales + (counter + st - s0 & 3) * 8;
                if (!wait(s_full(half), s_phase)) {
                    ok = false;
                    break;
                }
                s_phase ^= 1;
                tc_fence_after();
                const bool edge = pos0 + kKeys - 1 > min_pos ||
                                  (p.a.window > 0 && pos0 <= max_pos - p.a.window && pos0 + kKeys > p.a.sinks);
                const int hi = pos - pos0;                         // columns up to hi, and past lo or below sink
                const int lo = p.a.window > 0 ? hi - p.a.window : -1, sink = p.a.sinks - pos0;
                // the columns of 32 from c on that the row sees, as bits
                auto below = [](int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; };
                auto seen = [&](int c) { return below(hi + 1 - c) & (~below(lo + 1 - c) | below(sink - c)); };
                // two forms, with the mask and without
                auto weights = [&](auto tag) {
                constexpr bool EDGE = decltype(tag)::value;
                // the largest exponent: of each 16 keys the largest score, the factor not being negative
                float top = -INFINITY;
                uint32_t v[32], z[32];
                tmem_ld32_start(t_s, v);
#pragma unroll 1
                for (int c = 0; c < kKeys; c += 64) {
                    tmem_ld32_start(t_s + c + 32, z);
                    tmem_ld_wait(v);                               // both loads
                    auto most = [&](uint32_t (&x)[32], int from) {
                        if (EDGE) {
                            const uint32_t bits = seen(from);
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                if (!(bits >> k & 1)) x[k] = 0xff800000u;
                        }
#pragma unroll
                        for (int g = 0; g < 2; ++g) {
                            const float2 f = *reinterpret_cast<const float2 *>(sc + from / 16 + g);
                            float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
                            for (int k = 0; k < 16; k += 4) {
                                m0 = max3(m0, x[g * 16 + k], x[g * 16 + k + 1]);
                                m1 = max3(m1, x[g * 16 + k + 2], x[g * 16 + k + 3]);
                            }
                            top = fmaxf(top, fmaf(fmaxf(m0, m1), my_fac * f.x, f.y));
                        }
                    };
                    tmem_ld_wait(z);
                    most(v, c);
                    if (c + 64 < kKeys) tmem_ld32_start(t_s + c + 64, v);
                    most(z, c + 32);
                }
                tmem_ld32_start(t_s, v);                           // ahead of the weights
                if (__any_sync(0xffffffffu, top - ref > kTop)) {
                    const float to = top - ref > kTop ? top - kHead : ref;
                    const float f = ex2(ref - to);
                    ref = to;
                    sum *= f;
                    if (st > first_st) {
                        // out of the steps before is complete: this step's S was issued after it
#pragma unroll 1
                        for (int c = 0; c < D; c += 32) {
                            tmem_ld32(t_o + c, z);
#pragma unroll
                            for (int k = 0; k < 32; ++k) z[k] = __float_as_uint(__uint_as_float(z[k]) * f);
                            tmem_st32(t_o + c, z);
                        }
                    }
                }
                float part = 0.0f;
                auto weigh = [&](const uint32_t (&x)[32], int from) {
                    uint32_t pk[16];
                    const uint32_t bits = EDGE ? seen(from) : 0xffffffffu;
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        const float4 f4 = sc[from / 16 + g];
                        const float f = my_fac * f4.x, add = f4.y - ref;
                        const uint64_t ff = pair_of(f, f), aa = pair_of(add, add);
                        uint64_t ww = 0;
#pragma unroll
                        for (int i = 0; i < 16; i += 2) {
                            const int k = g * 16 + i;
                            float a, b;
                            unpair(fma2(pair_of(__uint_as_float(x[k]), __uint_as_float(x[k + 1])), ff, aa), a, b);
                            if (EDGE) {
                                if (!(bits >> k & 1)) a = -INFINITY;
                                if (!(bits >> (k + 1) & 1)) b = -INFINITY;
                            }
                            a = ex2(a), b = ex2(b);
                            ww = add2(ww, pair_of(a, b));
                            pk[k / 2] = pack_half2(a, b);
                        }
                        // a block that the row does not see adds nothing, whatever its scale
                        float w0, w1;
                        unpair(ww, w0, w1);
                        if (w0 + w1 != 0.0f) part = fmaf(w0 + w1, f4.z, part);
                    }
                    tmem_st16(t_s + from / 2, pk);                 // over scores that have been read
                };
#pragma unroll 1
                for (int c = 0; c < kKeys; c += 64) {
                    tmem_ld_wait(v);
                    tmem_ld32_start(t_s + c + 32, z);
                    weigh(v, c);
                    tmem_ld_wait(z);
                    if (c + 64 < kKeys) tmem_ld32_start(t_s + c + 64, v);
                    weigh(z, c + 32);
                }
                sum += part;
                };
                if (edge) weights(std::true_type{});
                else weights(std::false_type{});
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(p_ready(half));
            }
            if (!ok) break;
            counter += s1 - s0;
            if (!runs) {
                close_tile(idx);
                continue;
            }
            const bool joins = twice && s1 - s0 > 1;               // both halves have a part of these rows
            if (joins && half == 1) {
                // a row's two parts are in the same TMEM lane: the first half reads them both
                exchange[r] = make_float2(ref, sum);
                mbar_arrive(part_told);
                if (!wait(part_read, join_phase)) break;
                join_phase ^= 1;
                o_phase ^= 1;
                close_tile(idx);
                continue;
            }
            if (!wait(o_full(half), o_phase)) break;
            o_phase ^= 1;
            float f_here = 1.0f, f_there = 0.0f;
            if (half == 0) {
                // the other half's phases, so that its part can be waited for
                if (joins) {
                    if (!wait(o_full(1), other_phase)) break;
                    if (!wait(part_told, join_phase)) break;
                    join_phase ^= 1;
                    const float2 z = exchange[r];
                    const float m = fmaxf(ref, z.x);
                    f_here = ex2(ref - m), f_there = ex2(z.x - m);
                    sum = sum * f_here + z.y * f_there;
                    ref = m;
                }
                if (joins || !twice) other_phase ^= 1;
            }
            tc_fence_after();
            // 32 of the row's dims, of both parts
            auto read_out = [&](int c, float (&f)[32]) {
                uint32_t v[32];
                tmem_ld32(t_o + c, v);
#pragma unroll
                for (int k = 0; k < 32; ++k) f[k] = __uint_as_float(v[k]);
                if (joins) {
                    tmem_ld32(t_o + D + c, v);
#pragma unroll
                    for (int k = 0; k < 32; ++k) f[k] = fmaf(__uint_as_float(v[k]), f_there, f[k] * f_here);
                }
            };
            const bool has = exists;
            const long long at = (long long)(t.q0 + tok0 + r_tok) * p.a.n_heads + t.head * group + r_head;
            if (whole) {
                const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    float f[32];
                    read_out(c, f);
                    if (has) {
                        if constexpr (SHARED) kv_store_sums<D>(p.a, p.share, t.flags, at, c, f, 32, sum, ref);
                        else store(at, c, f, inv);
                    }
                }
                if (joins) {
                    tc_fence_before();
                    mbar_arrive(part_read);
                }
                if (!SHARED && has && p.a.lse)
                    p.a.lse[at] = sum == 0.0f ? -INFINITY : (ref + __log2f(sum)) * 0.6931471805599453f;
            } else {
                // a tile that CTAs from..to share: each leaves its part, in slot 1 the first of them, in slot 0
                // the others; the last of them to come adds them up
                // a part: D / 4 planes of a float4 a row, so that a warp's rows are one run, then (M, l) of the rows
                constexpr int kPart = kTileRows * (D + 2);
                auto slot = [&](int c, bool first) { return p.parts + ((long long)c * 2 + first) * kPart; };
                const int row = base_row + r;
                float *mine = slot(blockIdx.x, opens);
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    float f[32];
                    read_out(c, f);
                    if (has)
#pragma unroll
                        for (int k = 0; k < 32; k += 4)
                            __stcg(reinterpret_cast<float4 *>(mine) + (c + k) / 4 * kTileRows + row,
                                   make_float4(f[k], f[k + 1], f[k + 2], f[k + 3]));
                }
                if (joins) {
                    tc_fence_before();
                    mbar_arrive(part_read);
                }
                if (has) __stcg(reinterpret_cast<float2 *>(mine + kTileRows * D) + row, make_float2(ref, sum));
                const int from = first_cta(t, ctas, total), to = last_cta(t, ctas, total);
                if (SHARED && p.share.defer) {                     // whoever reads the rows sums the parts
                    if (has && opens) p.share.where[t.flags & kKvOthers][at] = kv_where(kKvManyParts, row, from, to);
                    tc_fence_before();
                    close_tile(idx);
                    continue;
                }
                // the tile's threads: of the first half, or of both
                auto meet = [&]() {
                    const uint32_t bar = meet_bar(twice ? 0 : 1);
                    int &phase = meet_phase[twice ? 0 : 1];
                    mbar_arrive(bar);
                    const bool met = wait(bar, phase);
                    phase ^= 1;
                    return met;
                };
                if (!meet()) break;
                if (tid == 0) {
                    __threadfence();
                    const bool done = ticket(from, to);
                    misc[3] |= opens ? 2 : 1;
                    __threadfence();
                    misc[2] = done;
                }
                if (!meet()) break;
                const bool last = *reinterpret_cast<volatile int *>(misc + 2);
                if (!meet()) break;                                // misc[2] is read before it is written again
                if (last && has) {
                    auto ml_of = [&](int c) {
                        return __ldcg(reinterpret_cast<const float2 *>(slot(c, c == from) + kTileRows * D) + row);
                    };
                    float m = kRefStart, l = 0.0f;
#pragma unroll 4
                    for (int c = from; c <= to; ++c) {
                        const float2 z = ml_of(c);
                        const float top = fmaxf(m, z.x);
                        l = fmaf(z.y, ex2(z.x - top), l * ex2(m - top));
                        m = top;
                    }
                    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll 1
                    for (int d = 0; d < D; d += 32) {
                        float f[32];
#pragma unroll
                        for (int k = 0; k < 32; ++k) f[k] = 0.0f;
#pragma unroll 1
                        for (int c = from; c <= to; c += 2) {      // two parts on their way together
                            const bool two = c < to;
                            const float4 *a = reinterpret_cast<const float4 *>(slot(c, c == from)) + d / 4 * kTileRows + row;
                            const float4 *b = reinterpret_cast<const float4 *>(slot(c + two, false)) + d / 4 * kTileRows + row;
                            const float wa = ex2(ml_of(c).x - m), wb = two ? ex2(ml_of(c + 1).x - m) : 0.0f;
                            float4 x[8], y[8];
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                x[k] = __ldcg(a + k * kTileRows);
                                y[k] = two ? __ldcg(b + k * kTileRows) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                            }
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                f[4 * k] = fmaf(y[k].x, wb, fmaf(x[k].x, wa, f[4 * k]));
                                f[4 * k + 1] = fmaf(y[k].y, wb, fmaf(x[k].y, wa, f[4 * k + 1]));
                                f[4 * k + 2] = fmaf(y[k].z, wb, fmaf(x[k].z, wa, f[4 * k + 2]));
                                f[4 * k + 3] = fmaf(y[k].w, wb, fmaf(x[k].w, wa, f[4 * k + 3]));
                            }
                        }
                        if constexpr (SHARED) kv_store_sums<D>(p.a, p.share, t.flags, at, d, f, 32, l, m);
                        else store(at, d, f, inv);
                    }
                    if (!SHARED && p.a.lse) p.a.lse[at] = l == 0.0f ? -INFINITY : (m + __log2f(l)) * 0.6931471805599453f;
                }
            }
            tc_fence_before();
            close_tile(idx);
        }
    } else if (warp < kSoftWarps + kConvWarps) {
        // ------------------------------------------------------------ codes to operands
        // A lane takes 16-byte piece `piece` of rows row0 + 4 i (head dim 128) or + 8 i (64): a warp's load
        // covers whole rows, and eight lanes' stores hit eight different bank groups.
        constexpr int ROWS = D == 128 ? 4 : 8;                     // rows of a warp's load
        constexpr int LOADS = 32 / ROWS;                           // loads of a warp's 32 rows
        const int w = warp - kSoftWarps;
        const int piece = D == 128 ? (lane & 3) | (lane >> 4) << 2 : lane & 3;
        const int row_in = D == 128 ? (lane >> 2) & 3 : lane >> 2;
        uint4 kraw[LOADS], vraw[LOADS];
        int page[2];                                               // of the warp's two 16-key groups; -2: not needed
        auto pages_of = [&](const ManyTile &t, int st) {
            const int pos0 = block_of(t, st) * kKeys + w * 32;
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const int at = pos0 + 16 * g;
                const bool needed = at <= t.hi && at < t.len && (at + 15 >= t.lo || at < p.a.sinks);
                const long long row = SHARED ? t.pages : (long long)t.seq * p.b.max_blocks;
                page[g] = needed ? p.b.block_table[row + (at >> p.c.page_shift)] : -2;
            }
        };
        auto check = [&]() {
#pragma unroll
            for (int g = 0; g < 2; ++g)
                if (page[g] != -2 && (page[g] < 0 || page[g] >= p.c.n_pages)) {
                    kv_report(p.status);
                    page[g] = -2;
                }
        };
        // where the warp's two groups of 16 keys begin in K, for this lane, and how many keys they hold
        struct Groups {
            const uint8_t *at[2];
            int rows[2];
        };
        const long long to_v = p.c.v - p.c.k;
        const long long row_step = ROWS * p.c.token_stride;
        const long long lane_at = row_in * p.c.token_stride + piece * 16;
        auto locate = [&](const ManyTile &t, int st) {
            Groups gr;
            const int pos0 = block_of(t, st) * kKeys + w * 32;
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const int at = pos0 + 16 * g;
                gr.rows[g] = page[g] >= 0 ? t.len - at : 0;
                gr.at[g] = p.c.k + (long long)page[g] * p.c.page_stride + t.head * p.c.head_stride +
                           (at & ((1 << p.c.page_shift) - 1)) * p.c.token_stride + lane_at;
            }
            return gr;
        };
        auto load = [&](const Groups &gr, long long to, uint4 (&raw)[LOADS]) {
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const uint8_t *src = gr.at[g] + to;
#pragma unroll
                for (int i = 0; i < LOADS / 2; ++i, src += row_step)
                    raw[g * (LOADS / 2) + i] = row_in + ROWS * i < gr.rows[g] ? ldg_stream_v4(src) : make_uint4(0, 0, 0, 0);
            }
        };
        float ks = 0.0f, vs = 0.0f;
        bool there = false;
        auto load_scales = [&](const ManyTile &t) {                // lanes 0 and 1: of the warp's two groups
            there = lane < 2 && page[lane & 1] >= 0;
            if (there) {
                const long long i = (long long)page[lane & 1] * Hk + t.head;
                ks = __ldg(p.c.k_scale + i);
                vs = __ldg(p.c.v_scale + i);
            }
        };
        ManyTile t;
        int st = 0, s1 = 0, idx = 0;
        bool more = false;
        auto open = [&]() {
            const PlannedTile *next = open_tile(idx);
            more = next != nullptr;
            if (more) t = next->t, st = next->s0, s1 = next->s1;
            close_tile(idx++);
        };
        // K a step ahead of V: S of the next step is wanted before this step's out.  Raw codes are loaded as
        // soon as their registers are free, a step ahead of their conversion.
        auto emit_k = [&](int c) {
            const int stg = c % L::kStages, ph = (c / L::kStages) & 1;
            if (!wait(k_empty(stg), ph ^ 1)) return false;
            uint8_t *dst = smem + L::kK + stg * L::kOperand;
            if (p.a.dtype == 0) convert_codes<KT, D, false>(kraw, dst, w * 32 + row_in, piece);
            else convert_codes<KT, D, true>(kraw, dst, w * 32 + row_in, piece);
            if (lane < 2)                                          // no page: weight 0 whatever the scores
                scales[(c & 3) * 8 + w * 2 + lane] =
                    there ? make_float4(ks, __log2f(vs), 1.0f / vs, 0.0f) : make_float4(0.0f, -INFINITY, 0.0f, 0.0f);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(k_full(stg));
            return true;
        };
        Groups gk = {};
        bool more_twice = false;                                   // the mode of the step that K's registers hold
        // the registers of K: the step after the one last loaded, if any
        auto advance = [&]() {
            if (++st == s1) open();
            if (more) pages_of(t, st);
        };
        auto load_k = [&]() {
            check();
            gk = locate(t, st);
            more_twice = same_rows(t);
            load(gk, 0, kraw);
            load_scales(t);
        };
        open();
        bool have_v = more;                                        // step c of the loop below exists
        if (more) {
            pages_of(t, st);
            load_k();
            load(gk, to_v, vraw);
        }
        bool twice = more_twice;
        if (more) {
            advance();
            if (!emit_k(0)) have_v = false;
            if (more) load_k();
        }
        for (int c = 0; have_v; ++c) {
            const bool have_k = more;                              // K of step c + 1 is in the registers
            const bool next_twice = more_twice;
            auto do_k = [&]() {
                if (!have_k) return true;
                advance();
                if (!emit_k(c + 1)) return false;
                if (more) load_k();
                return true;
            };
            const Groups after = gk;
            // The same rows twice: the other half waits for K.  Two halves of rows: K's place is free only once
            // the second half's S is done, V's before.
            if (twice && !do_k()) break;
            const int stg = c % L::kStages, ph = (c / L::kStages) & 1;
            if (!wait(v_empty(stg), ph ^ 1)) break;
            convert_codes<KT, D, false>(vraw, smem + L::kV + stg * L::kOperand, w * 32 + row_in, piece);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(v_full(stg));
            have_v = have_k;
            if (have_v) load(after, to_v, vraw);
            if (!twice && !do_k()) break;
            twice = next_twice;
        }
    }
    if (warp == kSoftWarps + kConvWarps) {
        // ------------------------------------------------------------ MMA issuer
        // S in the activations' type, its sign that of the scale (bit 13 negates Q): exponents then rise with scores
        const uint32_t idesc_s = make_idesc_f16(p.a.dtype, kHalfRows, kKeys) | (p.a.scale < 0.0f ? 1u << 13 : 0u);
        const uint32_t idesc_o = make_idesc_f16(0, kHalfRows, D) | 1u << 16;      // V is MN-major
        const uint32_t sm = smem_u32(smem);
        const uint32_t k_desc = (uint32_t)smem_desc_sw128(0u), v_desc = (uint32_t)desc_mn_sw128(0u, L::kBlockBytes);
        const uint32_t hi = (uint32_t)(smem_desc_sw128(0u) >> 32);
        int counter = 0, p_phase[2] = {0, 0}, q_phase[2] = {0, 0};
        auto scores = [&](int half, int stg) {
            mma_scores<L::kBlocks>(tmem + half * 128, k_desc + ((sm + L::kQ + half * L::kOperand) >> 4),
                                   k_desc + ((sm + L::kK + stg * L::kOperand) >> 4), hi, idesc_s);
            commit_elected(s_full(half));
        };
        auto output = [&](int half, int stg, bool fresh) {
            mma_output(tmem + 256 + half * D, tmem + half * 128, v_desc + ((sm + L::kV + stg * L::kOperand) >> 4), hi,
                       idesc_o, fresh ? 0u : 1u);
        };
        auto q_wait = [&](int half) {
            const int phase = q_phase[half];
            q_phase[half] ^= 1;
            return look(q_full(half), phase);
        };
        auto q_done = [&](int half) { commit_elected(q_empty(half)); };
        // MMAs run in the order they are issued: P is read before the next S of its half replaces it.
        auto run_tile = [&](int steps) {                           // two halves of rows, a step together
            for (int st = 0; st < steps; ++st, ++counter) {
                bool ok = true;
                const int stg = counter % L::kStages, ph = (counter / L::kStages) & 1;
                if (st == 0) {
                    ok &= look(k_full(stg), ph);
                    for (int h = 0; h < 2; ++h) {
                        ok &= q_wait(h);
                        tc_fence_after();
                        scores(h, stg);
                        if (steps == 1) q_done(h);
                    }
                    commit_elected(k_empty(stg));
                }
                const int nstg = (counter + 1) % L::kStages, nph = ((counter + 1) / L::kStages) & 1;
                for (int h = 0; h < 2; ++h) {
                    ok &= look(p_ready(h), p_phase[h]);
                    p_phase[h] ^= 1;
                    if (h == 0) ok &= look(v_full(stg), ph);
                    tc_fence_after();
                    output(h, stg, st == 0);
                    if (st + 1 == steps) commit_elected(o_full(h));
                    if (h == 1) commit_elected(v_empty(stg));
                    if (st + 1 < steps) {
                        if (h == 0) ok &= look(k_full(nstg), nph);
                        tc_fence_after();
                        scores(h, nstg);
                        if (h == 1) commit_elected(k_empty(nstg));
                        if (st + 2 == steps) q_done(h);
                    }
                }
                if (!all(ok)) return false;
            }
            return true;
        };
        auto run_same_rows = [&](int steps) {                      // the same rows twice, a half every other step
            for (int st = -2; st < steps; ++st) {
                const int h = st & 1;
                bool ok = true;
                if (st >= 0) {
                    const int c = counter + st, stg = c % L::kStages, ph = (c / L::kStages) & 1;
                    ok &= look(p_ready(h), p_phase[h]);
                    p_phase[h] ^= 1;
                    ok &= look(v_full(stg), ph);
                    tc_fence_after();
                    output(h, stg, st < 2);
                    if (st + 2 >= steps) commit_elected(o_full(h));
                    commit_elected(v_empty(stg));
                }
                if (st + 2 < steps) {
                    const int c = counter + st + 2, stg = c % L::kStages, ph = (c / L::kStages) & 1;
                    if (st < 0) ok &= q_wait(h);
                    ok &= look(k_full(stg), ph);
                    tc_fence_after();
                    scores(h, stg);
                    commit_elected(k_empty(stg));
                    if (st + 4 >= steps) q_done(h);
                }
                if (!all(ok)) return false;
            }
            counter += steps;
            return true;
        };
        for (int idx = 0;; ++idx) {
            const PlannedTile *next = open_tile(idx);
            if (!next) break;
            // the same in every lane, and known to be
            const int rows = __reduce_max_sync(0xffffffffu, next->t.rows);
            const int steps = __reduce_max_sync(0xffffffffu, next->s1 - next->s0);
            close_tile(idx);
            if (!(rows > half_rows ? run_tile(steps) : run_same_rows(steps))) break;
        }
        if (__any_sync(0xffffffffu, *abort_flag != 0)) {
            // leave with no product in flight
            commit_elected(drain);
            for (int i = 0; i < kDrainTries && !mbar_try_wait(drain, 0); ++i) {}
            __syncwarp();
        }
    } else if (warp == kSoftWarps + kConvWarps + 1) {
        // ------------------------------------------------------------ planner
        int pr = pair, hd = head, idx = 0, q_phase[2] = {0, 0};
        for (bool more = true; more;) {
            PlannedTile next = {};
            more = false;
            if (deal) {
                const int i = dealt(blockIdx.x, idx);
                if (i < pairs * Hk) {
                    next.t = tile_at(order[i / Hk], i % Hk);
                    next.s1 = next.t.steps;
                    more = true;
                }
            }
            while (!deal && pr < pairs) {
                next.t = tile_at(pr, hd);
                if (next.t.begin >= c1) break;
                if (++hd == Hk) hd = 0, ++pr;
                // this CTA's steps of the tile
                next.s0 = (int)min(max(c0 - next.t.begin - kCost, 0LL), (long long)next.t.steps);
                next.s1 = (int)min(max(c1 - next.t.begin - kCost, 0LL), (long long)next.t.steps);
                if (next.s0 < next.s1) {
                    more = true;
                    break;
                }
            }
            if (!more) next.s1 = 0;
            if (idx >= kRing &&
                !wait(plan_empty(idx % kRing), (idx / kRing - 1) & 1))
                break;
            if (lane == 0) {
                plan[idx % kRing] = next;
                mbar_arrive(plan_full(idx % kRing));
            }
            __syncwarp();
            // its rows of Q: a half's tokens times the group's heads, 64 dims a box, rows in that order
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (!more || !half_runs(next, h)) continue;
                if (!wait(q_empty(h), q_phase[h] ^ 1)) {
                    more = false;
                    break;
                }
                q_phase[h] ^= 1;
                if (lane == 0 && !kv_holds(p.hold)) {
                    const int tok = next.t.q0 + (next.t.row0 + (same_rows(next.t) ? 0 : h * half_rows)) / group;
                    mbar_arrive_expect_tx(q_full(h), (uint32_t)(half_rows * D * 2));
                    for (int b = 0; b < L::kBlocks; ++b)
                        tma_load_3d(smem_u32(smem) + L::kQ + h * L::kOperand + b * L::kBlockBytes, &tm_q, q_full(h), b * 64,
                                    next.t.head * group, tok);
                }
                __syncwarp();
            }
            ++idx;
        }
        if (__any_sync(0xffffffffu, *abort_flag != 0) && !kv_holds(p.hold)) {
            // leave with no copy in flight: q_phase counts a half's copies
            for (int h = 0; h < 2; ++h)
                for (int i = 0; i < kDrainTries && !mbar_try_wait(q_full(h), q_phase[h] ^ 1); ++i) {}
            __syncwarp();
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (*abort_flag && tid == 0 && !misc[4] && !(SHARED && p.share.defer)) {
        // A CTA that gave a wait up has no results, but its tickets are counted: they are back at 0 after every
        // launch, also for a replay, whose tag is the same.  All out of shared memory: the loops have no register to
        // spare for what is needed here.
        const int n = misc[5];
        const long long all = pre[n] * Hk, shares = min((long long)grid, (all + kCost) / (1 + kCost));
        const long long from = s_cut[0], to = s_cut[1];
        for (int i = 0; i < 2 && from < to; ++i) {
            const long long at = i ? to - 1 : from;
            int pr = 0;
            while (pr + 1 < n && pre[pr + 1] * Hk <= at) ++pr;
            const ManyTile t = tile_at(pr, (int)((at - pre[pr] * Hk) / (pre[pr + 1] - pre[pr])));
            const long long s0 = max(from - t.begin - kCost, 0LL), s1 = min(to - t.begin - kCost, (long long)t.steps);
            const bool others = s0 < s1 && (i ? s0 == 0 && s1 < t.steps : s0 > 0);
            if (others && !(misc[3] >> i & 1)) ticket(first_cta(t, shares, all), last_cta(t, shares, all));
        }
    }
    if (warp == kSoftWarps + kConvWarps) tmem_dealloc(tmem, 512u);
}

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                   const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// q as (dim, head, token); a box is 64 dims of a kv head's group over a half's tokens.
cudaError_t encode_q(const DeviceInfo &dev, const KvAttentionArgs &a, int n_tokens, int head_dim, int group,
                     CUtensorMap *out) {
    if (dev.encode_tiled == nullptr) return cudaErrorNotSupported;
    const cuuint64_t dims[3] = {(cuuint64_t)head_dim, (cuuint64_t)a.n_heads, (cuuint64_t)n_tokens};
    const cuuint64_t strides[2] = {(cuuint64_t)head_dim * 2, (cuuint64_t)a.q_stride * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)group, (cuuint32_t)(kHalfRows / group)}, one[3] = {1, 1, 1};
    const CUresult r = reinterpret_cast<EncodeTiledFn>(dev.encode_tiled)(
        out, a.dtype == 0 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(a.q),
        dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
        CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <bool SHARED, int KT, int D>
cudaError_t launch(const CUtensorMap &q, const ManyParams &p, int grid, cudaStream_t s, bool pdl) {
    using L = ManySmem<D>;
    auto kern = many_rows_kernel<SHARED, KT, D>;
    const cudaError_t e = raise_smem_cap(reinterpret_cast<const void *>(kern), L::kEnd);
    if (e != cudaSuccess) return e;
    return kv_launch(kern, dim3(grid), dim3(kThreads), L::kEnd, s, pdl, q, p);
}

template <bool SHARED>
cudaError_t launch_many(const KvAttentionArgs &a, const KvCache &c, const KvBatch &batch, int row_limit,
                        const DeviceInfo &dev, cudaStream_t s, bool pdl, KvShare share) {
    const int group = a.n_heads / c.n_kv_heads, half_rows = kHalfRows / group * group;
    CUtensorMap q;
    cudaError_t e = encode_q(dev, a, batch.n_tokens, c.head_dim, group, &q);
    if (e != cudaSuccess) return e;
    static std::atomic<unsigned long long> launches{SHARED ? 0x7e57ab1f0000ull : 0x7e57ab1e0000ull};
    const KvEntry *entries = share.entries;
    constexpr int kMost = SHARED ? kMaxEntries : kMaxSeqs;
    for (int b0 = 0; b0 < batch.n_seqs; b0 += kMost) {
        KvBatch b = batch;
        if constexpr (SHARED) {
            share.entries = entries + b0;
        } else {
            b.block_table += (long long)b0 * b.max_blocks;
            b.kv_lens += b0;
            b.q_starts += b0;
        }
        b.n_seqs = std::min(kMost, batch.n_seqs - b0);
        // as many pairs as these sequences can have at most
        const long long pairs = (SHARED ? 2LL : 1LL) * b.n_tokens * group / (2 * half_rows) + b.n_seqs;
        for (long long first = 0; first < pairs; first += kMaxPairs) {
            // with a row limit the other kernel has seen to the rows that no sequence owns
            const bool mine = !SHARED && row_limit == 0 && first == 0;
            ManyParams p{a, c, b, row_limit, half_rows, mine && b0 == 0, mine && b0 + b.n_seqs == batch.n_seqs, (int)first,
                         nullptr, nullptr, 0, hold_copies(), dev.status, share};
            p.tickets = static_cast<unsigned long long *>(a.workspace);
            p.parts = reinterpret_cast<float *>(p.tickets + ((dev.sm_count + 1) & ~1));
            p.tag = (launches.fetch_add(1) * 0x9e3779b97f4a7c15ull) >> 16;
            if (p.tag == 0) p.tag = 1;
            const int grid = dev.sm_count;
            if (c.kv_dtype == kKvInt8)
                e = c.head_dim == 128 ? launch<SHARED, kKvInt8, 128>(q, p, grid, s, pdl)
                                      : launch<SHARED, kKvInt8, 64>(q, p, grid, s, pdl);
            else
                e = c.head_dim == 128 ? launch<SHARED, kKvE4m3, 128>(q, p, grid, s, pdl)
                                      : launch<SHARED, kKvE4m3, 64>(q, p, grid, s, pdl);
            if (e != cudaSuccess) return e;
        }
    }
    return cudaSuccess;
}

}  // namespace

bool kv_attention_many_at_once(const KvBatch &batch, int group) {
    const long long rows = 2LL * batch.n_tokens * group;
    return batch.n_seqs <= kMaxEntries && rows / (2 * (kHalfRows / group * group)) + batch.n_seqs <= kMaxPairs;
}

cudaError_t launch_kv_attention_many(const KvAttentionArgs &a, const KvCache &c, const KvBatch &batch, int row_limit,
                                     const DeviceInfo &dev, cudaStream_t s, bool pdl, const KvShare *share) {
    return share ? launch_many<true>(a, c, batch, row_limit, dev, s, pdl, *share)
                 : launch_many<false>(a, c, batch, row_limit, dev, s, pdl, KvShare{});
}

long long kv_attention_many_workspace(int head_dim, const DeviceInfo &dev) {
    return (long long)((dev.sm_count + 1) & ~1) * 8 + (long long)dev.sm_count * 2 * kTileRows * (head_dim + 2) * 4;
}

}  // namespace w4a16
