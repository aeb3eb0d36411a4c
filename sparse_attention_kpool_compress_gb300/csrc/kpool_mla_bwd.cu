// Backward pass of the sparse attention over the selection (kpool_mla.cu): the
// gradients of the queries and of the latent rows, which are keys and values.
// For query row t and head h, over the row's token list J(t), with the log-sum
// lse and the output o that the forward pass left and their gradients:
//
//   p_j     = exp(scale * q[t, h, :] . c[j, :] - lse[t, h])
//   delta   = sum_d do[t, h, d] o[t, h, d] - dlse[t, h]
//   ds_j    = scale * p_j * (do[t, h, :] . c[j, :] - delta)
//   dq[t, h, :]  = sum_j ds_j c[j, :]
//   dc[j, :]    += ds_j q[t, h, :] + p_j do[t, h, :]
//
// Design (one persistent CTA per SM, 28 warps, rows handed out by an atomic
// counter, the last first).  Q and dO of a row are stacked, eight heads of one and
// the same eight of the other in turn: X [128 x 512].  Per block of 64 listed tokens
// C [64 x 512], in tensor memory:
//   [S; dP]  [128 x 64]    = X . C^T                       (A, B K-major)
//   dQ^T     [512 x 64]   += C^T . dS^T                    (A MN-major, B K-major)
//   dC^T     [512 x 64]    = X^T . [dS; P]                 (A, B MN-major)
// so every MMA has M = 128 and N = 64, one copy of X serves both orders, and so
// does one tile [dS; P] [128 x 64].  Heads in eights put the score and the dP of a
// (head, token) into one thread's registers (a 16x256b load has lanes r and r + 8),
// so P and dS need no exchange; lse is known, so no maximum and no sum either.
//   warp 0       control: rows, and per block a record with its token ids
//   warp 1       MMA issuer (the loop in all lanes, one issues)
//   warp 2       X (TMA), ahead into L2
//   warps 4-11   lse and delta of a row, while X lands; P and dS; after a row's last
//                block, dQ
//   warps 12-19  dC^T from tensor memory, added to the FP32 sums in L2
//   warps 20-27  loaders: the tokens' latent rows by 16-byte cp.async, a pair of
//                warps per slot of 128 columns
// The MMAs' order is: a block's scores; the last part of the last block's dC, while P
// and dS are made; dQ, which frees the slots one by one; three parts of dC, while the
// next block's rows land.  dC goes in four parts through three slots of tensor memory.
// P and dS are rounded to BF16, the type of the MMAs' operands (2^-8 of each at most);
// everything that is summed, is summed in FP32.
//
// Two kernels more: in front, cleared sums; behind, the sums rounded to BF16.  Where rows
// are few (half the SMs or less), a row's blocks are cut into even runs, one for each CTA,
// whose FP32 dQ the last kernel adds up.
//
// What bounds it: three costs that overlap in part.  10 * 64 * 512 FLOP a (row, token), in
// MMAs of N = 64 that take 48 cycles for their operands where the tensor pipe needs 32: 80
// of them are 3860 of a block's 8000 cycles.  2 KB added into L2 for each (row, token), at 6.0
// to 6.3 TB/s where the sums fit L2 (64 MB; random rows of 256 MB 3.7).  The path to shared
// memory, 73% busy (operands 48%; each dC value goes through it twice).  32768 rows of up to
// 2051 tokens take 27.9 ms (764 TFLOP/s, 4.8 TB/s of additions), of which the MMAs as they
// are take 13.4 and the additions alone 22; 131072 rows run at the same rate where
// neighbours choose much the same pools (114 ms), and at 4.3 TB/s with pools chosen at random
// (127 ms).  What neighbours have in common could be summed on chip before it is added: lists
// nest below the budget, and beyond it two rows of that choice list 57% (4096 keys) to 68%
// (32768) of the tokens of two rows apart.  This kernel adds each row by itself: two rows' X
// (256 KB) do not fit a CTA.
// Steps on 8192 rows: four sums warps with 4-byte additions 9.8 ms; through shared memory
// with 16-byte additions 7.5; eight such warps, X ahead into L2 6.8; the first parts of dC
// moved behind dQ 6.65; X in quarters, token ids read ahead 6.47; X given up in quarters
// 6.40; lse and delta in this kernel instead of one in front 6.34 (3001 packed tokens 431
// -> 401 us).  Slower: bulk reductions from shared memory (8.0 to 8.6), direct 4-byte
// additions by eight warps (6.7), waits polled by one lane (11.1) or without suspending
// (9.3).
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include "kpool_internal.h"
#include "kpool_mla_rows.cuh"
#include "kpool_ptx.cuh"

namespace kpool {
namespace {

constexpr int kH = 64;                  // heads
constexpr int kDc = 512;                // latent width
constexpr int kBT = 64;                 // listed tokens per block
constexpr int kThreads = 896;
constexpr int kGradWarp0 = 4, kGradWarps = 8;      // P and dS, dQ
constexpr int kSumWarp0 = kGradWarp0 + kGradWarps, kSumWarps = 8;
constexpr int kLoaderWarp0 = kSumWarp0 + kSumWarps, kLoaderWarps = 8;
static_assert(32 * (kLoaderWarp0 + kLoaderWarps) == kThreads, "warps");
constexpr int kGroup = 8192;            // eight rows of X: 8 chunks of 64 columns, 1 KB each
constexpr int kChunk = kBT * 128;       // 64 latent columns of a block
constexpr int kSlots = 4;               // 128 columns each
constexpr int kSlot = 2 * kChunk;
constexpr int kParts = 4;               // dQ^T and dC^T in parts of 128 latent columns
constexpr int kFirst = 3;               // parts of dC^T before the next block's scores
constexpr int kSumSlots = 3;
constexpr int kInfoSlots = 4;
constexpr uint64_t kTimeoutNs = 2000000000ull;
constexpr int kTmemCols = 512;          // dQ^T: 0..255, [S; dP]: 256..319, dC^T parts: 320..511
constexpr int kTmemS = 256, kTmemSum = 320;

// shared memory (from a 1024-byte aligned base)
constexpr int kOffX = 0;
constexpr int kOffC = kOffX + 16 * kGroup;
constexpr int kOffP = kOffC + kSlots * kSlot;          // [dS; P]: 16 groups of eight rows, 1 KB each
constexpr int kStage = 16 * 128;                       // 16 tokens x 32 columns of dC, a sums warp
constexpr int kOffStage = kOffP + 128 * 128;
constexpr int kOffInfo = kOffStage + kSumWarps * kStage;
constexpr int kOffTok = kOffInfo + kInfoSlots * 32;    // token ids [kInfoSlots][64]
constexpr int kOffBar = kOffTok + kInfoSlots * kBT * 4;
enum {
    BX_FULL = 0, BX_EMPTY = BX_FULL + kParts, BC_FULL = BX_EMPTY + kParts, BC_EMPTY = BC_FULL + kSlots, BS_FULL = BC_EMPTY + kSlots, BP_FULL, BP_EMPTY,
    BQ_FULL, BQ_EMPTY, BD_FULL, BD_EMPTY = BD_FULL + kSumSlots, BI_FULL = BD_EMPTY + kSumSlots,
    BI_EMPTY = BI_FULL + kInfoSlots, BDRAIN = BI_EMPTY + kInfoSlots, NBARS
};
constexpr int kOffMisc = kOffBar + NBARS * 8;          // [0] tmem base, [1] abort flag
constexpr int kSmemBytes = kOffMisc + 16 + 1024;       // and alignment slack
static_assert(kSmemBytes <= 232448, "shared memory over the per-block limit");

// workspace: header (ints: row counter, status; where rows are cut, the blocks of a run),
// the runs' dQ, sums
constexpr int kHeadInts = 256, kHeadRuns = 64;
constexpr int kMaxSms = 160;            // that a workspace has room for
constexpr int kMaxSplit = 64;           // runs of a row
static_assert(kHeadRuns + kMaxSms <= kHeadInts, "a word for each run");

struct Params {
    RowLists rows;
    const uint16_t *q, *kv, *o, *d_o;
    const float *lse, *d_lse;
    uint16_t *dq;
    float *acc;                 // [Tk, 512]: the latent rows' gradients
    int split;                  // runs of a row (1: rows are whole)
    float *part;                // [T * split, 64, 512]: dQ of the runs
    float scale, c_scale;       // softmax scale, and that * log2(e)
    int *ws;
    uint64_t wait_limit_ns;
};

// One block of a row.
struct BInfo {
    int t, b, nb, ksteps;       // b-th of nb blocks of a row, or of a run of row t
    uint32_t mask[2];           // bit r of mask[r / 32]: listed token r is valid
    int pad[2];
};
static_assert(sizeof(BInfo) == 32, "BInfo slot");

// Operand tiles whose groups of eight rows lie `group` bytes apart.
__device__ __forceinline__ uint64_t desc_k(uint32_t saddr, uint32_t group)
{
    return (ptx::smem_desc_sw128(saddr) & ~(0x3FFFull << 32)) | (static_cast<uint64_t>(group >> 4) << 32);
}

__device__ __forceinline__ uint64_t desc_mn(uint32_t saddr, uint32_t chunk, uint32_t group)
{
    return (ptx::smem_desc_mn_sw128(saddr, chunk) & ~(0x3FFFull << 32)) | (static_cast<uint64_t>(group >> 4) << 32);
}

// X: eight rows x 128 columns of q or d_o, as two chunks of 64 columns.
__device__ __forceinline__ void load_group(uint32_t dst, const void *desc, uint32_t bar, int row, int chunk)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(desc), "r"(bar), "r"(0), "r"(row), "r"(chunk)
        : "memory");
}

__device__ __forceinline__ void prefetch_l2(const void *from, uint32_t bytes)
{
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(from), "r"(bytes) : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void red_add(float *to, const float4 &v)
{
    asm volatile("red.relaxed.gpu.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(to), "f"(v.x), "f"(v.y), "f"(v.z),
                 "f"(v.w)
                 : "memory");
}

// Sum of the products of eight BF16 pairs.
__device__ __forceinline__ float dot8(const uint4 &x, const uint4 &y)
{
    const uint32_t a[4] = {x.x, x.y, x.z, x.w}, b[4] = {y.x, y.y, y.z, y.w};
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        s = fmaf(__uint_as_float(a[i] << 16), __uint_as_float(b[i] << 16), s);
        s = fmaf(__uint_as_float(a[i] & 0xFFFF0000u), __uint_as_float(b[i] & 0xFFFF0000u), s);
    }
    return s;
}

__device__ __forceinline__ void st_shared(uint32_t saddr, uint32_t v)
{
    asm volatile("st.shared.b32 [%0], %1;" ::"r"(saddr), "r"(v) : "memory");
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&b);
}

// (kPoll, for short limits, is a constant of its own: looked up at each wait it costs the
// 1111 lists of 333 tokens 8 of 219 us.)
template <bool kCut, bool kPoll>
__global__ void __launch_bounds__(kThreads, 1)
    sparse_mla_bwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_do,
                          const __grid_constant__ Params p)
{
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sbase = ptx::smem_u32(smem);
    const uint32_t sX = sbase + kOffX, sC = sbase + kOffC, sP = sbase + kOffP;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + kOffBar);
    auto bar = [&](int i) { return ptx::smem_u32(&bars[i]); };
    uint32_t *misc = reinterpret_cast<uint32_t *>(smem + kOffMisc);
    BInfo *info = reinterpret_cast<BInfo *>(smem + kOffInfo);
    int *toks = reinterpret_cast<int *>(smem + kOffTok);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kParts; ++i) {
            ptx::mbar_init(bar(BX_FULL + i), 1);
            ptx::mbar_init(bar(BX_EMPTY + i), 1);
        }
        for (int i = 0; i < kSlots; ++i) {
            ptx::mbar_init(bar(BC_FULL + i), 2);    // the slot's two loader warps
            ptx::mbar_init(bar(BC_EMPTY + i), 1);
        }
        ptx::mbar_init(bar(BS_FULL), 1);
        ptx::mbar_init(bar(BP_FULL), kGradWarps);
        ptx::mbar_init(bar(BP_EMPTY), 1);
        ptx::mbar_init(bar(BQ_FULL), 1);
        ptx::mbar_init(bar(BQ_EMPTY), kGradWarps);
        for (int i = 0; i < kSumSlots; ++i) {
            ptx::mbar_init(bar(BD_FULL + i), 1);
            ptx::mbar_init(bar(BD_EMPTY + i), kSumWarps);
        }
        for (int i = 0; i < kInfoSlots; ++i) {
            ptx::mbar_init(bar(BI_FULL + i), 1);
            ptx::mbar_init(bar(BI_EMPTY + i), 2 + kGradWarps + kSumWarps + kLoaderWarps);
        }
        ptx::mbar_init(bar(BDRAIN), 1);
        misc[1] = 0u;
        ptx::fence_mbar_init();
    }
    if (warp == 1) {
        ptx::tmem_alloc(ptx::smem_u32(&misc[0]), kTmemCols);
        ptx::tmem_relinquish();
        ptx::tc_fence_before();
    }
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = misc[0];
    const Sync sy{reinterpret_cast<volatile uint32_t *>(&misc[1]), p.ws + 1, p.wait_limit_ns, kPoll};
    // the cleared sums and counter of the kernel in front
    ptx::grid_dependency_wait();

    if (warp == 0) {
        // ---------------- control: rows and their blocks ----------------
        bool ok = true;
        int g = 0, run = blockIdx.x;    // blocks published; this CTA's run (of cut rows)
        while (ok) {
            int t = -1, b0 = 0;
            if (kCut) {
                if (run < 0) break;
                t = run / p.split;
            } else {
                if (lane == 0 && !*sy.abort_flag) t = p.rows.T - 1 - atomicAdd(p.ws, 1);
                t = __shfl_sync(kFull, t, 0);
                if (t < 0) break;
            }
            const RowMsg m = row_msg(p.rows, t, lane);
            int nb = max(1, (m.n_slots + kBT - 1) / kBT);
            if (kCut) {
                const int per = (nb + p.split - 1) / p.split;
                b0 = (run - t * p.split) * per;
                nb = max(0, min(nb - b0, per));
                if (lane == 0) p.ws[kHeadRuns + run] = nb;
                run = -1;
            }
            for (int b = 0; b < nb; ++b, ++g) {
                const int j0 = (b0 + b) * kBT;
                const int t0 = token_of(p.rows, m, j0 + 2 * lane), t1 = token_of(p.rows, m, j0 + 2 * lane + 1);
                // validity word w (tokens 32w .. 32w + 31) from lanes 16w .. 16w + 15
                uint32_t mw = ((t0 >= 0 ? 1u : 0u) | (t1 >= 0 ? 2u : 0u)) << (2 * (lane & 15));
                mw |= __shfl_xor_sync(kFull, mw, 1);
                mw |= __shfl_xor_sync(kFull, mw, 2);
                mw |= __shfl_xor_sync(kFull, mw, 4);
                mw |= __shfl_xor_sync(kFull, mw, 8);
                const int is = g % kInfoSlots;
                ok = wait_bar_warp(bar(BI_EMPTY + is), ((g / kInfoSlots) & 1) ^ 1, sy);
                if (!ok) break;
                *reinterpret_cast<int2 *>(toks + is * kBT + 2 * lane) = make_int2(t0, t1);
                if ((lane & 15) == 0) info[is].mask[lane >> 4] = mw;
                if (lane == 0) {
                    info[is].t = t;
                    info[is].b = b;
                    info[is].nb = nb;
                    info[is].ksteps = max(1, (min(kBT, m.n_slots - j0) + 15) / 16);
                }
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(bar(BI_FULL + is));
            }
        }
        // end of the block stream for every consumer
        const int is = g % kInfoSlots;
        if (ok && wait_bar_warp(bar(BI_EMPTY + is), ((g / kInfoSlots) & 1) ^ 1, sy) && lane == 0) {
            info[is].t = -1;
            ptx::mbar_arrive(bar(BI_FULL + is));
        }
    } else if (warp == 2) {
        // ---------------- X ----------------
        if (lane == 0) {
            ptx::tma_prefetch_desc(&tm_q);
            ptx::tma_prefetch_desc(&tm_do);
        }
        int sent = 0;                   // pieces of X so far
        for (int g = 0;; ++g) {
            const int is = g % kInfoSlots;
            if (!wait_bar_warp(bar(BI_FULL + is), (g / kInfoSlots) & 1, sy)) break;
            const int t = info[is].t, b = info[is].b;
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar(BI_EMPTY + is));
            if (t < 0) break;
            if (b > 0) continue;
            // (known some blocks ahead: into L2 meanwhile)
            if (lane < 3)
                prefetch_l2((lane == 0 ? p.q : lane == 1 ? p.d_o : p.o) + static_cast<int64_t>(t) * kH * kDc, kH * kDc * 2);
            // in pieces of 128 columns: the scores take them in turn, and the last block's dC has
            // given them up in turn
            bool ok = true;
            for (int i = 0; i < kParts && ok; ++i) {
                ok = wait_bar_warp(bar(BX_EMPTY + i), (sent / kParts & 1) ^ 1, sy);
                if (!ok) break;
                if (lane == 0) ptx::mbar_arrive_expect_tx(bar(BX_FULL + i), 16 * kGroup / kParts);
                __syncwarp();
                if (lane < 16)
                    load_group(sX + lane * kGroup + i * 2048, (lane & 1) ? &tm_do : &tm_q, bar(BX_FULL + i),
                               t * kH + 8 * (lane >> 1), 2 * i);
                ++sent;
            }
            if (!ok) break;
        }
        // no load of X may still be in flight when the CTA ends: a wait of its own for the
        // last pieces, bounded by the default limit and blind to the abort flag
        for (int n = max(0, sent - kParts); n < sent; ++n) {
            const uint64_t t0 = ptx::globaltimer();
            while (!ptx::mbar_try_wait(bar(BX_FULL + n % kParts), n / kParts & 1))
                if (ptx::globaltimer() - t0 > kTimeoutNs) break;
        }
    } else if (warp == 1) {
        // ---------------- MMA issuer ----------------
        constexpr uint32_t idesc = ptx::make_idesc(1u, 128, 64);
        const bool one = ptx::elect_one();
        int g = 0;
        uint32_t c_ph = 0, x_ph = 0, q_ph = 0, nd = 0;      // nd: parts of dC so far
        bool any = false, rest = false;                     // rest: the last block's dC lacks its last part
        // parts of dC^T = X^T . [dS; P]
        auto sum_parts = [&](int part0, int part1, bool last) {
#pragma unroll 1
            for (int part = part0; part < part1; ++part, ++nd) {
                const uint32_t s = nd % kSumSlots;
                if (!wait_bar_warp(bar(BD_EMPTY + s), ((nd / kSumSlots) & 1) ^ 1, sy)) return false;
                ptx::tc_fence_after();
                if (one) {
                    const uint64_t ad = desc_mn(sX + part * 2048, 1024, kGroup), bd = desc_mn(sP, 1024, 1024);
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        ptx::mma_bf16(tmem + kTmemSum + s * 64, ad + kk * (2 * kGroup / 16), bd + kk * 128,
                                      idesc | ptx::kIdescAMajorMN | ptx::kIdescBMajorMN, kk > 0);
                    ptx::mma_commit(bar(BD_FULL + s));
                    // (these columns of X have served the row)
                    if (last) ptx::mma_commit(bar(BX_EMPTY + part));
                }
            }
            if (part0 > 0 && one) ptx::mma_commit(bar(BP_EMPTY));
            return true;
        };
        for (;;) {
            const int is = g % kInfoSlots;
            if (!wait_bar_warp(bar(BI_FULL + is), (g / kInfoSlots) & 1, sy)) break;
            const BInfo in = info[is];
            __syncwarp();
            if (one) ptx::mbar_arrive(bar(BI_EMPTY + is));
            if (rest && (in.t < 0 || in.b == 0)) {
                // the row ends: the next one's X waits for this
                if (!sum_parts(kFirst, kParts, true)) break;
                rest = false;
            }
            if (in.t < 0) break;
            bool ok = true;
            // (the last block's scores were read before its P was complete)
            for (int sl = 0; sl < kSlots; ++sl) {
                ok = (in.b > 0 || wait_bar_warp(bar(BX_FULL + sl), x_ph, sy)) && wait_bar_warp(bar(BC_FULL + sl), c_ph, sy);
                if (!ok) break;
                ptx::tc_fence_after();
                if (one) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint64_t ad = desc_k(sX + (2 * sl + h) * 1024, kGroup);
                        const uint64_t bd = desc_k(sC + sl * kSlot + h * kChunk, 1024);
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            ptx::mma_bf16(tmem + kTmemS, ad + 2 * kk, bd + 2 * kk, idesc, (sl | h | kk) != 0);
                    }
                }
                any = true;
            }
            if (!ok) break;
            if (in.b == 0) x_ph ^= 1;
            if (one) ptx::mma_commit(bar(BS_FULL));
            // the last part of the last block's dC while P and dS are made
            if (rest && !sum_parts(kFirst, kParts, false)) break;
            if (!wait_bar_warp(bar(BP_FULL), g & 1, sy)) break;
            if (in.b == 0 && !wait_bar_warp(bar(BQ_EMPTY), q_ph ^ 1, sy)) break;
            ptx::tc_fence_after();
            if (one) {
                for (int sl = 0; sl < kSlots; ++sl) {
                    const uint64_t ad = desc_mn(sC + sl * kSlot, kChunk, 1024), bd = desc_k(sP, 2048);
                    for (int kk = 0; kk < in.ksteps; ++kk)
                        ptx::mma_bf16(tmem + sl * 64, ad + kk * 128, bd + 2 * kk, idesc | ptx::kIdescAMajorMN,
                                      in.b > 0 || kk > 0);
                    ptx::mma_commit(bar(BC_EMPTY + sl));
                }
                if (in.b == in.nb - 1) ptx::mma_commit(bar(BQ_FULL));
            }
            if (in.b == in.nb - 1) q_ph ^= 1;
            if (!sum_parts(0, kFirst, in.b == in.nb - 1)) break;
            rest = true;
            c_ph ^= 1;
            ++g;
        }
        if (any) {
            if (one) ptx::mma_commit(bar(BDRAIN));
            const uint64_t t0 = ptx::globaltimer();
            while (!ptx::mbar_try_wait(bar(BDRAIN), 0))
                if (ptx::globaltimer() - t0 > kTimeoutNs) break;
        }
    } else if (warp >= kGradWarp0 && warp < kSumWarp0) {
        // ---------------- P and dS, dQ ----------------
        const int sub = warp & 3, half = (warp - kGradWarp0) >> 2;
        const int grp = 2 * sub + half;                    // heads 8 grp .. 8 grp + 7
        const int head = 8 * grp + (lane >> 2);
        const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * sub) << 16);
        const uint32_t s_at = lanes + (static_cast<uint32_t>(16 * half) << 16) + kTmemS;
        // a thread has tokens 8 j + 2 (lane % 4) and the next, for j = 0 .. 7
        const uint32_t row = sP + 2 * grp * 1024 + (lane >> 2) * 128 + (lane & 3) * 4;
        float lse = 0.f, delta = 0.f;
        uint32_t q_ph = 0;
        for (int g = 0;; ++g) {
            const int is = g % kInfoSlots;
            if (!wait_bar_warp(bar(BI_FULL + is), (g / kInfoSlots) & 1, sy)) break;
            const BInfo in = info[is];
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar(BI_EMPTY + is));
            if (in.t < 0) break;
            if (in.b == 0) {
                // the row's statistics, while X lands: every lane sums this warp's heads in turn
                const int64_t row0 = static_cast<int64_t>(in.t) * kH;
                const float l = p.lse[row0 + head];
                lse = l == -INFINITY ? INFINITY : l * 1.4426950408889634f;     // (no token: no probability)
                delta = p.d_lse != nullptr ? -p.d_lse[row0 + head] : 0.f;
                const uint4 *o = reinterpret_cast<const uint4 *>(p.o) + (row0 + 8 * grp) * 64 + lane;
                const uint4 *d = reinterpret_cast<const uint4 *>(p.d_o) + (row0 + 8 * grp) * 64 + lane;
#pragma unroll 1
                for (int h = 0; h < 8; h += 2) {
                    uint4 x[4], y[4];                      // two heads, two halves each
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        x[i] = o[h * 64 + 32 * i];
                        y[i] = d[h * 64 + 32 * i];
                    }
                    float v[2];
#pragma unroll
                    for (int k = 0; k < 2; ++k) v[k] = dot8(x[2 * k], y[2 * k]) + dot8(x[2 * k + 1], y[2 * k + 1]);
#pragma unroll
                    for (int w = 16; w > 0; w >>= 1) {
                        v[0] += __shfl_xor_sync(kFull, v[0], w);
                        v[1] += __shfl_xor_sync(kFull, v[1], w);
                    }
                    if ((lane >> 2) == h) delta += v[0];
                    if ((lane >> 2) == h + 1) delta += v[1];
                }
            }
            if (!wait_bar_warp(bar(BS_FULL), g & 1, sy)) break;
            ptx::tc_fence_after();
            uint32_t r[32];
            ptx::tmem_ld16x256_x8(s_at, r);
            ptx::tmem_ld_wait(r);
            uint32_t w2[8], ds2[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t m = in.mask[j >> 2] >> (8 * (j & 3) + 2 * (lane & 3));
                float w[2], ds[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float x = ptx::ex2_approx(fmaf(__uint_as_float(r[4 * j + e]), p.c_scale, -lse));
                    const float y = x * ((__uint_as_float(r[4 * j + 2 + e]) - delta) * p.scale);
                    const bool v = (m >> e) & 1u;
                    w[e] = v ? x : 0.f;
                    ds[e] = v ? y : 0.f;
                }
                w2[j] = pack_bf16(w[0], w[1]);
                ds2[j] = pack_bf16(ds[0], ds[1]);
            }
            // the last block's dC has read [dS; P]
            if (!wait_bar_warp(bar(BP_EMPTY), (g & 1) ^ 1, sy)) break;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t at = row + ((j ^ (lane >> 2)) << 4);
                st_shared(at, ds2[j]);
                st_shared(at + 1024, w2[j]);
            }
            ptx::tc_fence_before();
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar(BP_FULL));
            if (in.b == in.nb - 1) {
                if (!wait_bar_warp(bar(BQ_FULL), q_ph, sy)) break;
                q_ph ^= 1;
                ptx::tc_fence_after();
                uint16_t *out = p.dq + static_cast<int64_t>(in.t) * kH * kDc + 32 * sub + lane;
#pragma unroll 1
                for (int part = 2 * half; part < 2 * half + 2; ++part)
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) {
                        uint32_t v[32];
                        ptx::tmem_ld32(lanes + part * 64 + hh * 32, v);
                        ptx::tmem_ld_wait(v);
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const int64_t at = static_cast<int64_t>(hh * 32 + i) * kDc + part * 128;
                            if (kCut) {
                                p.part[static_cast<int64_t>(blockIdx.x) * kH * kDc + 32 * sub + lane + at] = __uint_as_float(v[i]);
                            } else {
                                const __nv_bfloat16 b = __float2bfloat16_rn(__uint_as_float(v[i]));
                                out[at] = *reinterpret_cast<const uint16_t *>(&b);
                            }
                        }
                    }
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(bar(BQ_EMPTY));
            }
        }
    } else if (warp >= kSumWarp0 && warp < kLoaderWarp0) {
        // ---------------- sums of dC ----------------
        // Four warps take the first 32 tokens of each part, four the others.
        const int sub = warp & 3, tok0 = 32 * ((warp - kSumWarp0) >> 2);
        const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * sub) << 16) + kTmemSum + tok0;
        const uint32_t stage = sbase + kOffStage + (warp - kSumWarp0) * kStage;
        uint32_t nd = 0;
        bool ok = true;
        for (int g = 0; ok; ++g) {
            const int is = g % kInfoSlots;
            ok = wait_bar_warp(bar(BI_FULL + is), (g / kInfoSlots) & 1, sy);
            if (!ok || info[is].t < 0) break;
            // the tokens whose sums this lane adds to: 4 k + lane / 8
            int tk[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) tk[k] = toks[is * kBT + tok0 + 4 * k + (lane >> 3)];
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar(BI_EMPTY + is));
            for (int part = 0; part < kParts; ++part, ++nd) {
                const uint32_t s = nd % kSumSlots;
                ok = wait_bar_warp(bar(BD_FULL + s), (nd / kSumSlots) & 1, sy);
                if (!ok) break;
                ptx::tc_fence_after();
                float *to = p.acc + part * 128 + 32 * sub + 4 * (lane & 7);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t v[16];
                    tmem_ld16(lanes + s * 64 + h * 16, v);
                    if (h == 1) {
                        ptx::tc_fence_before();
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive(bar(BD_EMPTY + s));
                    }
                    // (lanes are latent columns: through shared memory, so that eight lanes
                    // add 128 bytes of a token's row, 16 each)
#pragma unroll
                    for (int i = 0; i < 16; ++i) st_shared(stage + i * 128 + lane * 4, v[i]);
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float4 x = ptx::ld_shared_v4(stage + k * 512 + lane * 16);
                        const int tok = tk[4 * h + k];
                        if (tok >= 0) red_add(to + static_cast<int64_t>(tok) * kDc, x);
                    }
                    __syncwarp();
                }
            }
        }
    } else if (warp >= kLoaderWarp0) {
        // ---------------- loaders ----------------
        const int sl = (warp - kLoaderWarp0) >> 1;                 // the slot of this pair
        const int t64 = ((warp - kLoaderWarp0) & 1) * 32 + lane;   // 0..63 within the pair
        const int k = t64 & 15;                                    // 16-byte piece of the slot's 256 bytes
        const char *kvb = reinterpret_cast<const char *>(p.kv) + sl * 256 + k * 16;
        const uint32_t dst = sC + sl * kSlot + (k >> 3) * kChunk;
        bool ok = true;
        uint32_t c_ph = 0;
        for (int g = 0;; ++g) {
            const int is = g % kInfoSlots;
            ok = wait_bar_warp(bar(BI_FULL + is), (g / kInfoSlots) & 1, sy);
            if (!ok || info[is].t < 0) break;
            int tk[kBT / 4];                                       // rows t64 / 16 + 4 i
#pragma unroll
            for (int i = 0; i < kBT / 4; ++i) tk[i] = toks[is * kBT + (t64 >> 4) + 4 * i];
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar(BI_EMPTY + is));
            ok = wait_bar_warp(bar(BC_EMPTY + sl), c_ph ^ 1, sy);
            if (!ok) break;
#pragma unroll
            for (int i = 0; i < kBT / 4; ++i) {
                const int r = (t64 >> 4) + 4 * i;
                ptx::cp_async16(dst + r * 128 + (((k & 7) ^ (r & 7)) << 4),
                                kvb + (tk[i] >= 0 ? static_cast<int64_t>(tk[i]) * (kDc * 2) : 0), tk[i] >= 0 ? 16u : 0u);
            }
            ptx::cp_async_commit();
            ptx::cp_async_wait_all();
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar(BC_FULL + sl));
            c_ph ^= 1;
        }
        ptx::cp_async_wait_all();
    }

    __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, kTmemCols);
    }
}

// In front: cleared sums, counter and status.
__global__ void __launch_bounds__(256) clear_kernel(float4 *acc, int64_t n, int *ws)
{
    const int64_t first = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x;
    const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
    ptx::grid_dependents_launch();
    if (first < 64) ws[first] = 0;
    for (int64_t i = first; i < n; i += step) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
}

__device__ __forceinline__ uint4 round8(const float4 &a, const float4 &b)
{
    return make_uint4(pack_bf16(a.x, a.y), pack_bf16(a.z, a.w), pack_bf16(b.x, b.y), pack_bf16(b.z, b.w));
}

// The sums of the latent rows' gradients, rounded to BF16, and the runs' dQ added up: eight
// values a thread.
__global__ void __launch_bounds__(256) round_kernel(const float4 *acc, uint4 *dkv, int64_t n, const float4 *part,
                                                    uint4 *dq, int64_t n_dq, int split, const int *runs)
{
    ptx::grid_dependency_wait();
    const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
    const int64_t first = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x;
    for (int64_t i = first; i < n; i += step) dkv[i] = round8(acc[2 * i], acc[2 * i + 1]);
    constexpr int kRow = kH * kDc / 8;
    for (int64_t i = first; i < n_dq; i += step) {
        const int64_t t = i / kRow, at = i % kRow;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
        for (int64_t r = t * split; r < (t + 1) * split; ++r) {
            if (runs[r] == 0) break;                       // (runs without blocks come last)
            const float4 x = part[2 * (r * kRow + at)], y = part[2 * (r * kRow + at) + 1];
            a.x += x.x; a.y += x.y; a.z += x.z; a.w += x.w;
            b.x += y.x; b.y += y.y; b.z += y.z; b.w += y.w;
        }
        dq[i] = round8(a, b);
    }
}

template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), int grid, int threads, int smem, cudaStream_t s, const A &...args)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Runs of a row, where rows are at most half of the SMs: as many as fill them, and no more
// than the longest list has blocks.  More rows are whole, one to a CTA at a time, so that a
// last round that is not full costs a whole one (76 rows 88 us, 77 to 152 148, 153 275).  (2051 tokens a row, us a call in a graph, cut and
// whole: 1 row 29 and 145, 16 rows 37 and 147, 38 rows 57 and 147, 76 rows, in two runs
// each, 92 and 148.)
int runs(int64_t T, int64_t slots, int sms)
{
    if (T == 0 || 2 * T > sms) return 1;
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({sms / T, (slots + kBT - 1) / kBT, kMaxSplit})));
}

}  // namespace

// (Neither the device that a caller sizes its workspace on nor the lists' width is known
// here: room for as many runs as there can be.)
size_t sparse_mla_bwd_workspace_need(int64_t T, int64_t Tk)
{
    const int64_t n = T * runs(T, int64_t(kMaxSplit) * kBT, kMaxSms);
    return kHeadInts * 4 + (n > T ? static_cast<size_t>(n) * kH * kDc * 4 : 0) +
           static_cast<size_t>(Tk) * kDc * 4;
}

// (Few rows need more than many, which are not cut: the most that T rows or fewer need, so
// that a workspace for the largest batch serves the smaller ones.)
size_t sparse_mla_bwd_workspace_bytes(int64_t T, int64_t Tk)
{
    size_t most = sparse_mla_bwd_workspace_need(T, Tk);
    for (int64_t t = std::min<int64_t>(T, kMaxSms / 2); t > 0; --t)
        most = std::max(most, sparse_mla_bwd_workspace_need(t, Tk));
    return most;
}

int run_sparse_mla_bwd(const SparseMlaArgs &a, const SparseMlaGrad &g, cudaStream_t s)
{
    uint8_t *ws = static_cast<uint8_t *>(a.workspace);
    Params p{};
    p.rows = row_lists(a);
    p.q = static_cast<const uint16_t *>(a.q);
    p.kv = static_cast<const uint16_t *>(a.kv);
    p.o = static_cast<const uint16_t *>(a.o);
    p.d_o = static_cast<const uint16_t *>(g.d_o);
    p.lse = a.lse;
    p.d_lse = g.d_lse;
    p.dq = static_cast<uint16_t *>(g.dq);
    const int sms = std::min(num_sms(), kMaxSms);
    // (pools list a token once at most)
    p.split = runs(a.T, a.tok_idx != nullptr ? a.W : std::min<int64_t>(a.Tk, static_cast<int64_t>(a.Kp) * a.kpool + a.kpool - 1),
                   sms);
    p.part = reinterpret_cast<float *>(ws + kHeadInts * 4);
    p.acc = p.part + (p.split > 1 ? a.T * p.split * kH * kDc : 0);
    p.scale = a.scale;
    p.c_scale = static_cast<float>(static_cast<double>(a.scale) * 1.4426950408889634);
    p.ws = reinterpret_cast<int *>(ws);
    p.wait_limit_ns = get_wait_limit_ns();
    const int64_t rows = a.T * kH, n_acc = a.Tk * (kDc / 4);
    clear_kernel<<<static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>((n_acc + 1023) / 1024, 8 * sms))), 256, 0, s>>>(
        reinterpret_cast<float4 *>(p.acc), n_acc, p.ws);
    KPOOL_CUDA_CHECK(cudaGetLastError());
    if (a.T > 0) {
        CUtensorMap mq, mdo;
        int rc = encode_bf16_groups_tmap(&mq, a.q, static_cast<uint64_t>(rows));
        if (rc) return rc;
        rc = encode_bf16_groups_tmap(&mdo, g.d_o, static_cast<uint64_t>(rows));
        if (rc) return rc;
        const bool poll = p.wait_limit_ns < kPollBelowNs;
        const auto kernel = p.split > 1 ? (poll ? sparse_mla_bwd_kernel<true, true> : sparse_mla_bwd_kernel<true, false>)
                                        : (poll ? sparse_mla_bwd_kernel<false, true> : sparse_mla_bwd_kernel<false, false>);
        KPOOL_CUDA_CHECK(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes));
        KPOOL_CUDA_CHECK(launch_after(kernel, static_cast<int>(p.split > 1 ? a.T * p.split : std::min<int64_t>(sms, a.T)),
                                      kThreads, kSmemBytes, s, mq, mdo, p));
    }
    const int64_t n = a.Tk * (kDc / 8), n_dq = p.split > 1 ? a.T * (kH * kDc / 8) : 0;
    if (std::max(n, n_dq) > 0)
        KPOOL_CUDA_CHECK(launch_after(
            round_kernel, static_cast<int>(std::min<int64_t>((std::max(n, n_dq) + 255) / 256, 8 * sms)), 256, 0, s,
            reinterpret_cast<const float4 *>(p.acc), static_cast<uint4 *>(g.dkv), n, reinterpret_cast<const float4 *>(p.part),
            static_cast<uint4 *>(g.dq), n_dq, p.split, static_cast<const int *>(p.ws + kHeadRuns)));
    return KPOOL_OK;
}

}  // namespace kpool
