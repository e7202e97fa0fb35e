// rows_attn.cu — attention of rows of queries over packed 2-bit caches on the
// 5th-generation tensor cores: cross attention (queries of one length against
// cached states of another, per sequence) and single-token decode over a
// prefix that groups of sequences share.
//
// The rows of one unit are queries that read the same keys: the G query heads
// of a KV head times the Nq queries of a sequence (cross), or times the
// sequences of a group (shared prefix). With khat and vhat the dequantized
// keys and values of "QuantWM: Training-Free 2-bit KV Cache Quantization for
// Stable Video World Models" ("1. QSAC") and u = qP its compensation
// ("2. PSAC"),
//
//   s_rt = (q_r . khat_t + u_r . a_t) sm_scale,   o_r = sum_t softmax_t(s_r) vhat_t.
//
// with tcgen05: S [128 rows x 128 keys] = Q . Khat^T + U . A^T into TMEM, the
// softmax by a thread per row, P back into the columns of S, O += P . Vhat in
// TMEM. Operands are fp16 as in the chunk kernel: Khat = fp16(code s +
// fp16(z + mu)), Vhat = fp16(code s + z) with exact codes, one rounding per fp16
// operation; queries scaled per row by a power of two, which leaves bf16 values
// exact; U = fp16 of an fp32 product of the bf16 query with P in two bf16
// halves; P = fp16(p).
//
// Two softmax groups of four warps keep the tensor core and the exponentials
// busy in turn. With more than 128 rows (WIDE, units of 256 rows) each group has
// 128 rows of its own, and every dequantized tile serves both. With fewer, both
// groups have the same 128 rows and take the tiles alternately, each with its
// own S, O, maximum and sum, joined when the unit's rows are written; rows that
// do not exist cost their warps nothing. (A transposed form, keys in the tile's
// rows and the queries in as few columns as there are, was built and measured
// first: its per-column maxima and sums cost about 13,000 warp instructions per
// 128 x 128 scores, against 4,000 here, and the tensor core's time, which it
// saves for few rows, is not what bounds either.)
//
// Softmax: p = 2^(s log2e - m_r + 7) against a running maximum m_r that may
// trail the true one by 2^7: p stays below 2^14 and keeps 21 binary orders of
// normal fp16 below the maximum, and O is rescaled only when a row's scores pass
// m_r by more than that. m_r is a whole number: every rescaling is by an exact
// power of two, and p's rounding does not depend on where the work is cut.
//
// Warp roles of a CTA (one per SM): 8 softmax warps; 8 warps that dequantize
// keys and 8 for values (they also load the unit's queries: all of them 256
// rows, the value warps 128), so that the waits and loads of one overlap the
// arithmetic of the other; one warp that
// issues the MMAs, polling both groups; one thread that copies packed tiles to
// shared memory. Registers are traded between the roles' warpgroups.
//
// Work: the key tiles of all units form one list (source, sequence, KV head,
// row block, tile), of which every CTA takes an equal contiguous part, found
// from the lengths on the device (a captured call replays with other lengths).
// A unit that a part's border cuts is written in pieces (unnormalised rows,
// maximum, sum) and merged by a second kernel.
//
// Every wait is bounded by an SM-clock budget; on expiry the CTA's abort flag
// ends the other waits, the workspace's first word is set, the rows of the
// CTA's remaining part become NaN and the kernel ends. No row is finished from
// operands that are not there: producers whose wait failed go on over whatever
// their stages hold, but only after the flag is up, and a unit's rows are
// written as numbers only where the flag is still down after the wait for
// their last product; the next product that starts on the same columns waits
// for the softmax warps of the group, which arrive no more once their own wait
// has failed.
//
// Measured on a B200 (cold caches): 4,680 queries x 4,096 keys x 40 heads 759 us,
// 533 TFLOP/s, 0.32 of the bf16 GEMM rate; x 512 keys 153 us; 32 rows (8
// continuations of 4 heads) over 32,768 shared keys 65 us. Bound: the softmax
// and the hand-overs between the roles. A tile takes about 8,300 cycles for two
// groups of 128 rows (softmax 4,000, of them 2,048 the exponentials; tensor core
// 2,100) and 5,000 with up to 128 rows (keys 2,900), a unit 20,000 more for its
// queries, first maxima and output rows.
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "internal.h"
#include "mbarrier.cuh"
#include "packed_tile.cuh"
#include "row_division.h"
#include "umma.cuh"

namespace kv2 {
namespace {

constexpr int kKeys = 128;             // keys per tile
constexpr int kRows = 128;             // rows per softmax group (TMEM lanes)
constexpr float kBias = 7.0f;          // p = 2^(x) with x = s log2e - m + kBias
constexpr float kTrail = 7.0f;         // a score this far above the running maximum moves it
// A unit begins with kLead positions of the work list that hold no tile: its
// query rows, first maxima and output rows take about as long as that many key
// tiles, so parts with many short units get fewer tiles.
constexpr int kLead = 2;
constexpr int kForceTile = 4;

struct RowsSource {
  const uint32_t* k_code;
  const uint32_t* v_code;
  const uint32_t* k_sz;
  const uint32_t* v_sz;
  const void* cidx;
  const uint16_t* psac;
  const uint16_t* psac_scale;
  const uint16_t* cent;
  const float* P;
  const int32_t* table;
  const int32_t* lens;      // [B] (null: max_len for every sequence)
  const int32_t* q_lens;    // [B] (null: Nq)
  int B, M, r, cap, page, gshift, psac_fmt, max_len, Nq;
};

struct RowsParams {
  RowsSource src[2];
  int nsrc, H_kv, H_q;
  RowDivision by_group;     // by G = H_q / H_kv
  __device__ int per_head(int row) const { return int(by_group(uint32_t(row))); }
  const uint16_t* Q;        // bf16 [rows of (b, i)][H_q][D]
  void* out;                // null: whole units go to dir_o / dir_ml
  int out_dtype;
  float scale_log2, q_sign; // |sm_scale| log2(e), and sm_scale's sign, which the queries take
  int* err;
  long long* total;         // workspace: length of the work list
  long long* base;          // workspace: first position of every sequence, [src 0 | src 1]
  int4* cta;                // workspace: {source, sequence, unit in the sequence, first tile in the unit} per CTA
  float* part_o;            // pieces [CTA][2][N][D], slot 0: continues a unit, 1: begins one
  float2* part_ml;          // [CTA][2][N] running maximum and sum
  float* dir_o;             // whole units [source][rows][D]
  float2* dir_ml;
  long long dir_rows;       // rows per source of dir_*
  const float* split_part;  // the second source's results from the split decode kernel (null: from this one)
  int splits;
  uint32_t none;            // 0 (see the producers' release of a packed tile)
  unsigned long long budget;
  int force_timeout;        // tests: 1 every CTA's first wait expires, 2 + c: CTA c's wait for its packed tile kForceTile
};

// D channels; WIDE: units of 256 rows, else of 128
template <int D, bool WIDE>
struct RCfg {
  static constexpr int X = WIDE ? 2 : 1, N = kRows * X;
  static constexpr int SW = 8, PW = 8, CH = D / 2;           // warps per role; channels per producer thread
  static constexpr int kValueWarp = SW + PW, kMmaWarp = SW + 2 * PW, kLoadWarp = kMmaWarp + 1;
  // (whole warpgroups, so that they can trade registers)
  static constexpr int kThreads = 32 * (SW + 2 * PW + 4);
  // registers per thread by role, in all the launch's threads times kRegs
  static constexpr int kRegs = 72, kRegsSoft = 88, kRegsProd = 64, kRegsIssue = 72;
  static_assert(SW * kRegsSoft + 2 * PW * kRegsProd + 4 * kRegsIssue <= (SW + 2 * PW + 4) * kRegs, "register split");
  // stages of keys, values and packed tiles. One of keys is enough: with WIDE
  // units the keys of tile t + 1 are multiplied a softmax after they could first
  // be written, else the scores' columns are free as late. A third packed tile
  // hides the copies' latency instead (128 rows over 32,768 keys, 8 KV heads: 61
  // us against 65 us with two stages of keys and two packed tiles).
  static constexpr int KS = 1, VS = WIDE ? 1 : 2, RS = 3;
  // packed tile: codes of keys and values, scale and zero words, ids, PSAC
  // (fp16, or int8 codes and from RAW_PSC on the tokens' scales)
  static constexpr int RAW_VC = kKeys * D / 4, RAW_KZ = 2 * RAW_VC, RAW_VZ = RAW_KZ + kKeys * D / 8;
  static constexpr int RAW_IX = RAW_VZ + kKeys * D / 8, RAW_PS = RAW_IX + 2 * kKeys, RAW_PSC = RAW_PS + kKeys * 16;
  static constexpr int RAW_BYTES = RAW_PS + kKeys * 32;
  static constexpr int Q_BYTES = kRows * D * 2, U_BYTES = kRows * 32, K_BYTES = kKeys * D * 2, A_BYTES = kKeys * 32;
  static constexpr int V_BYTES = kKeys * D * 2;
  static constexpr uint32_t OFF_K = 0;
  static constexpr uint32_t OFF_V = OFF_K + KS * K_BYTES;
  static constexpr uint32_t OFF_Q = OFF_V + VS * V_BYTES;
  static constexpr uint32_t OFF_A = OFF_Q + X * Q_BYTES;
  static constexpr uint32_t OFF_RAW = OFF_A + KS * A_BYTES;
  static constexpr uint32_t OFF_U = OFF_RAW + RS * RAW_BYTES;
  static constexpr uint32_t OFF_FRAG = OFF_U + X * U_BYTES;             // P fragments [D/16][2][2][32] uint2
  static constexpr uint32_t OFF_SCR = OFF_FRAG + D / 16 * 2 * 2 * 32 * 8;   // row scales, ring of 4 units
  static constexpr uint32_t OFF_ML = OFF_SCR + 4 * N * 4;                    // maxima and sums of both groups, float2 [2][kRows]
  // output rows on their way out of WIDE units, 2 KB a softmax warp
  static constexpr uint32_t OFF_STG = OFF_ML + 2 * kRows * 8;
  static constexpr uint32_t OFF_BAR = OFF_STG + (WIDE ? SW * 2048 : 0);
  static constexpr uint32_t SMEM = OFF_BAR + 288 + 1024;
  static constexpr uint32_t kTmemCols = 512;           // S of both groups, O of both groups
  // Q, U, Khat, A K-major; Vhat by channels
  static constexpr uint32_t kIdQK = make_idesc(0, 0, 0, kKeys, kRows);
  static constexpr uint32_t kIdPV = make_idesc(0, 0, 1, D, kRows);
  static_assert(SMEM <= 232448, "shared memory of one CTA");
};
// barrier slots (bytes from OFF_BAR)
constexpr uint32_t B_KFULL = 0, B_KEMPTY = 16, B_VFULL = 32, B_VEMPTY = 48, B_SFULL = 64, B_PFULL = 96,
                   B_PDONE = 128, B_QFULL = 192, B_QEMPTY = 200, B_FINAL = 208, B_NEVER = 216,
                   B_TMEM = 224, B_ABORT = 228, B_RFULL = 232, B_REMPTY = 256;

__device__ __forceinline__ void bar_sync(int id, int count) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(count) : "memory");
}
__device__ __forceinline__ bool bar_or(int id, int count, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\tbar.red.or.pred p, %2, %3, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(r)
      : "r"(uint32_t(v)), "r"(id), "r"(count)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void ldsm_x4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
// d += A B, m16n8k16, bf16 operands, fp32 sums
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// whether the barrier's phase of this parity has completed (no wait)
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t phase) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred P1;\n\tmbarrier.test_wait.parity.shared::cta.b64 P1, [%1], %2;\n\t"
      "selp.b32 %0, 1, 0, P1;\n\t}\n"
      : "=r"(done)
      : "r"(bar), "r"(phase)
      : "memory");
  return done != 0;
}
// 16 bytes global -> shared by the asynchronous copy (zeros when !ok)
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// e with |x| < 2^e (finite x; -126 at least), and 2^e
__device__ __forceinline__ int exp_above(float x) { return int((__float_as_uint(x) >> 23) & 0xffu) - 126; }
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }
// this warpgroup's registers per thread: R, of the launch's LAUNCHED
template <int R, int LAUNCHED>
__device__ __forceinline__ void set_regs() {
  if constexpr (R > LAUNCHED) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
  if constexpr (R < LAUNCHED) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}
// one lane of the warp
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(r));
  return r != 0;
}
// ---------------------------------------------------------------------------
// the work list: every unit is kLead positions, then one per key tile
// ---------------------------------------------------------------------------

// first position of CTA c of C over T positions, and the CTA that holds position u
__device__ __forceinline__ long long quot(long long a, long long b) {       // of non-negative numbers
  return ((a | b) >> 32) == 0 ? static_cast<long long>(uint32_t(a) / uint32_t(b)) : a / b;
}
__device__ __forceinline__ long long part_begin(long long T, int c, int C) { return quot(T * c, C); }
__device__ __forceinline__ int part_of(long long u, long long T, int C) { return int(quot((u + 1) * C - 1, T)); }

// keys and queries of a sequence
__device__ __forceinline__ int seq_len(const RowsSource& s, int b) {
  return s.lens ? min(max(s.lens[b], 0), s.max_len) : s.max_len;
}
__device__ __forceinline__ int seq_queries(const RowsSource& s, int b) {
  return s.q_lens ? min(max(s.q_lens[b], 0), s.Nq) : s.Nq;
}
// tiles per unit (an empty sequence has one masked tile: its rows become zero)
// and row blocks of a sequence (its rows fit in 30 bits)
__device__ __forceinline__ int tiles_of(int len) { return max(1, (len + kKeys - 1) / kKeys); }
template <int N>
__device__ __forceinline__ int blocks_of(int ql, int G) { return (ql * G + N - 1) / N; }

// a place in the list; every role of a CTA walks the same segments
template <int N>
struct Walk {
  int left;                 // positions from the unit's first tile to the part's end
  int src, b, h, rb, j;     // row block rb of KV head h of sequence b, next tile j
  int len, ql;
  __device__ void load(const RowsParams& p) {
    len = seq_len(p.src[src], b);
    ql = seq_queries(p.src[src], b);
  }
  __device__ int count() const { return min(tiles_of(len), left) - j; }
  __device__ bool more() const { return j < left; }
  __device__ void next(const RowsParams& p) {
    left -= tiles_of(len) + kLead;
    j = 0;
    if (left <= 0) return;
    const int G = p.H_q / p.H_kv;
    if (++rb < blocks_of<N>(ql, G)) return;
    rb = 0;
    if (++h < p.H_kv) return;
    h = 0;
    do {
      if (++b == p.src[src].B) {
        b = 0;
        ++src;
      }
      load(p);
    } while (ql == 0);
  }
};

// The list's length and this CTA's place in it, by one warp: the positions of
// 32 sequences at a time, summed by shuffles.
template <int N>
__device__ void plan(const RowsParams& p, int lane, Walk<N>& w) {
  const int G = p.H_q / p.H_kv, C = gridDim.x, c = blockIdx.x;
  long long T = 0, lo = 0, hi = 0;
  for (int pass = 0; pass < 2; ++pass) {
    long long at = 0;
    bool found = false;
    for (int s = 0; s < p.nsrc && !found; ++s) {
      for (int b0 = 0; b0 < p.src[s].B && !found; b0 += 32) {
        const int b = b0 + lane;
        long long v = 0;
        if (b < p.src[s].B) {
          v = static_cast<long long>(tiles_of(seq_len(p.src[s], b)) + kLead) *
              blocks_of<N>(seq_queries(p.src[s], b), G) * p.H_kv;
        }
        long long inc = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long up = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += up;
        }
        if (pass == 0) {
          if (c == 0 && b < p.src[s].B) p.base[(s ? p.src[0].B : 0) + b] = at + inc - v;
        } else {
          const unsigned hit = __ballot_sync(0xffffffffu, at + inc > lo);
          if (hit) {
            const int l = __ffs(hit) - 1;
            w.src = s;
            w.b = b0 + l;
            const long long rem = lo - (at + __shfl_sync(0xffffffffu, inc - v, l));
            w.load(p);
            const int unit = tiles_of(w.len) + kLead, ub = int(quot(rem, unit)), in = int(rem - static_cast<long long>(ub) * unit);
            const int RB = blocks_of<N>(w.ql, G);
            w.h = ub / RB;
            w.rb = ub % RB;
            w.j = max(0, in - kLead);
            w.left = int(hi - (lo - in + kLead));
            found = true;
          }
        }
        at += __shfl_sync(0xffffffffu, inc, 31);
      }
    }
    if (pass == 0) {
      T = at;
      lo = part_begin(T, c, C);
      hi = part_begin(T, c + 1, C);
      if (c == 0 && lane == 0) *p.total = T;
      if (lo >= hi) return;
    }
  }
}

// ---------------------------------------------------------------------------
// producers
// ---------------------------------------------------------------------------

// W consecutive 32-bit words of shared memory
template <int W>
__device__ __forceinline__ void load_words(const uint8_t* src, uint32_t* w) {
  if constexpr (W == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(src);
    w[0] = v.x; w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < W; i += 4) {
      const uint4 v = *reinterpret_cast<const uint4*>(src + 4 * i);
      w[i] = v.x; w[i + 1] = v.y; w[i + 2] = v.z; w[i + 3] = v.w;
    }
  }
}

// eight channels: codes lc of a code word times s2 plus add, in fp16 pairs
__device__ __forceinline__ uint4 dequant8(uint32_t word, int lc, uint32_t s2, const uint32_t (&add)[4]) {
  const uint32_t x = field_both(word, lc), x8 = x >> 8;
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = hfma2(code_pair_f16(x, x8, i), s2, add[i]);
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// ---------------------------------------------------------------------------
template <int D, bool WIDE>
__global__ void __launch_bounds__(RCfg<D, WIDE>::kThreads, 1) rows_attn_kernel(const __grid_constant__ RowsParams p) {
  using Cfg = RCfg<D, WIDE>;
  constexpr int N = Cfg::N, SW = Cfg::SW, PW = Cfg::PW, KS = Cfg::KS, VS = Cfg::VS, CH = Cfg::CH;
  extern __shared__ uint8_t smem_raw[];
  // (by pointer arithmetic, so that accesses stay shared-memory accesses)
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sb = smem_u32(smem);
  const uint32_t bar = sb + Cfg::OFF_BAR;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Cfg::OFF_BAR + B_TMEM);
  volatile int* abort = reinterpret_cast<volatile int*>(smem + Cfg::OFF_BAR + B_ABORT);
  __shared__ Walk<N> walk_s;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = p.H_q / p.H_kv;

  if (tid == 32) {
    // one arrival per warp of the arriving role, or an MMA commit
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar + B_KFULL + 8 * i, PW);
      mbar_init(bar + B_KEMPTY + 8 * i, 1);
      mbar_init(bar + B_VFULL + 8 * i, PW);
      mbar_init(bar + B_VEMPTY + 8 * i, 1);
      mbar_init(bar + B_SFULL + 8 * i, 1);        // per softmax group
      mbar_init(bar + B_PFULL + 8 * i, SW / 2);
      mbar_init(bar + B_PDONE + 8 * i, 1);
    }
    for (int i = 0; i < Cfg::RS; ++i) {
      mbar_init(bar + B_RFULL + 8 * i, 1);
      mbar_init(bar + B_REMPTY + 8 * i, 2 * PW);
    }
    mbar_init(bar + B_QFULL, N / 16);
    mbar_init(bar + B_QEMPTY, 1);
    mbar_init(bar + B_FINAL, 1);
    mbar_init(bar + B_NEVER, 1);
    mbar_init_fence();
    *abort = 0;
  }
  if (warp == Cfg::kMmaWarp) tmem_alloc(smem_u32(tmem_slot), Cfg::kTmemCols);
  if (warp == 0) {
    Walk<N> w;
    w.left = w.src = w.b = w.h = w.rb = w.j = w.len = w.ql = 0;
    plan<N>(p, lane, w);
    if (lane == 0) {
      walk_s = w;
      p.cta[blockIdx.x] = make_int4(w.src, w.b, w.h * blocks_of<N>(w.ql, G) + w.rb, w.j);
    }
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  Walk<N> w = walk_s;

  if (warp >= Cfg::kMmaWarp) {
    set_regs<Cfg::kRegsIssue, Cfg::kRegs>();
    if (warp == Cfg::kMmaWarp) {
    // ================= MMA issue =================
    // The warp's control flow is made uniform by votes and shuffles, so that the
    // descriptors stay in uniform registers: eight MMAs issue in about 400
    // cycles, against 630 from a lane picked by its index. Both groups are
    // polled, so that neither waits for the other's softmax.
    constexpr uint32_t kIdQK = Cfg::kIdQK, kIdPV = Cfg::kIdPV;
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint64_t dK = make_sdesc(sb + Cfg::OFF_K, 16, 1024, kLayoutSW128);
    const uint64_t dA = make_sdesc(sb + Cfg::OFF_A, 128, 256, kLayoutNone);
    const uint64_t dV = make_sdesc(sb + Cfg::OFF_V, 16384, 1024, kLayoutSW128);
    const uint64_t dQ = make_sdesc(sb + Cfg::OFF_Q, 16, 1024, kLayoutSW128);
    const uint64_t dU = make_sdesc(sb + Cfg::OFF_U, 128, 256, kLayoutNone);
    auto ready = [&](uint32_t b, uint32_t phase) __attribute__((always_inline)) {
      return __all_sync(0xffffffffu, mbar_test(bar + b, phase)) != 0;
    };
    // a group's next tile: t counts the CTA's tiles, jj the part's tiles of the unit
    struct Cursor {
      Walk<N> w;
      int cnt, jj, t, seg;
      bool psac, pv;                             // pv: the tile's scores are issued, P . V is next
    } cur[2];
    auto settle = [&](Cursor& c) __attribute__((always_inline)) {   // to the unit that holds the tile
      for (;;) {
        c.cnt = __shfl_sync(0xffffffffu, c.w.more() ? c.w.count() : 0, 0);
        if (c.cnt == 0) return;
        if (c.jj < c.cnt) break;
        c.jj -= c.cnt;
        ++c.seg;
        c.w.next(p);
      }
      c.psac = __shfl_sync(0xffffffffu, p.src[c.w.src].r, 0) > 0;
    };
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      cur[x].w = w;
      cur[x].t = cur[x].jj = WIDE ? 0 : x;
      cur[x].seg = 0;
      cur[x].pv = cur[x].psac = false;
      settle(cur[x]);
    }
    int scores = 0;                               // tiles whose scores are issued (by the only group that takes them)
    unsigned long long since = clock64();
    bool ok = true;
    if (p.force_timeout == 1) ok = __all_sync(0xffffffffu, mbar_wait_or_abort(bar + B_NEVER, 0, p.budget, abort));
    while (ok && (cur[0].cnt || cur[1].cnt)) {
      bool moved = false;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        Cursor& c = cur[x];
        Cursor& o = cur[1 - x];
        if (c.cnt == 0) continue;
        const int k = WIDE ? c.t : c.t >> 1;      // the group's tiles before this one
        const uint32_t tS = tm + x * kKeys, tO = tm + 2 * kKeys + x * kRows;
        // with WIDE units, whether the other group is past this tile's step
        const bool other_s = !WIDE || o.cnt == 0 || o.t > c.t || (o.t == c.t && o.pv);
        const bool other_v = !WIDE || o.cnt == 0 || o.t > c.t;
        if (!c.pv) {
          const int s = c.t % KS;
          if (!WIDE && scores != c.t) continue;   // in the order of the tiles
          if (k > 0 && !ready(B_PDONE + 8 * x, (k - 1) & 1)) continue;     // P lies in the columns of S
          if (!ready(B_KFULL + 8 * s, (c.t / KS) & 1)) continue;
          if (!ready(B_QFULL, c.seg & 1)) continue;
          fence_after_sync();
          if (elect_one()) {
            const uint64_t a = dQ + uint64_t((WIDE ? x * Cfg::Q_BYTES : 0) >> 4), b = dK + uint64_t(s * Cfg::K_BYTES >> 4);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint64_t off = uint64_t(((kk >> 2) * 16384 + (kk & 3) * 32) >> 4);
              mma_f16(tS, a + off, b + off, kIdQK, kk > 0);
            }
            if (c.psac)
              mma_f16(tS, dU + uint64_t((WIDE ? x * Cfg::U_BYTES : 0) >> 4), dA + uint64_t(s * Cfg::A_BYTES >> 4), kIdQK, 1);
            mma_commit(bar + B_SFULL + 8 * x);
            if (other_s) {
              mma_commit(bar + B_KEMPTY + 8 * s);
              if (c.jj == c.cnt - 1) mma_commit(bar + B_QEMPTY);
            }
          }
          __syncwarp();
          ++scores;
          c.pv = true;
          moved = true;
        } else {
          const int s = c.t % VS;
          if (!ready(B_PFULL + 8 * x, k & 1)) continue;
          if (!ready(B_VFULL + 8 * s, (c.t / VS) & 1)) continue;
          fence_after_sync();
          if (elect_one()) {
            const bool first = c.jj < (WIDE ? 1 : 2);    // the group's first tile of the unit's part
            const uint64_t b = dV + uint64_t(s * Cfg::V_BYTES >> 4);
#pragma unroll
            for (int kk = 0; kk < kKeys / 16; ++kk)
              mma_f16_tmem_a(tO, tS + kk * 8, b + uint64_t(kk * 2048 >> 4), kIdPV, kk > 0 || !first);
            mma_commit(bar + B_PDONE + 8 * x);
            if (other_v) mma_commit(bar + B_VEMPTY + 8 * s);
          }
          __syncwarp();
          c.pv = false;
          c.t += WIDE ? 1 : 2;
          c.jj += WIDE ? 1 : 2;
          settle(c);
          moved = true;
        }
      }
      const unsigned long long now = clock64();
      if (moved) since = now;
      else if (__any_sync(0xffffffffu, *abort || now - since > p.budget)) {
        *abort = 1;
        ok = false;
      }
    }
    } else if (warp == Cfg::kLoadWarp) {
    // ================= packed tiles (one thread, bulk copies) =================
    if (lane == 0) {
      int t = 0;
      for (; w.more(); w.next(p)) {
        const RowsSource& s = p.src[w.src];
        const int cnt = w.count(), sz = (D >> s.gshift) * 4, id = s.M <= 256 ? 1 : 2;
        const int ps = s.psac_fmt == 1 ? s.r : 2 * s.r, psc = s.psac_fmt == 1 && s.r ? 2 : 0;
        bool out = false;
        for (int jj = 0; jj < cnt; ++jj, ++t) {
          const int st = t % Cfg::RS, tok = (w.j + jj) * kKeys;
          if (t >= Cfg::RS && !mbar_wait_or_abort(bar + B_REMPTY + 8 * st, (t / Cfg::RS - 1) & 1, p.budget, abort)) {
            out = true;
            break;
          }
          if (t == kForceTile && p.force_timeout == 2 + int(blockIdx.x)) {
            *abort = 1;
            out = true;
            break;
          }
          const uint32_t full = bar + B_RFULL + 8 * st, dst = sb + Cfg::OFF_RAW + st * Cfg::RAW_BYTES;
          // whole runs of 16 tokens (16-byte copies), within the capacity, which is a multiple of 16;
          // a tile never leaves its page
          const int n = (min(kKeys, w.len - tok) + 15) & ~15;
          if (n <= 0) {                           // an empty sequence's masked tile
            mbar_arrive(full);
            continue;
          }
          const size_t slot = cache_slot(s.table, s.page, p.H_kv, s.cap, w.b, w.h, tok);
          mbar_arrive_expect_tx(full, uint32_t(n) * uint32_t(D / 2 + 2 * sz + id + ps + psc));
          bulk_g2s(dst, s.k_code + slot * (D / 16), n * (D / 4), full);
          bulk_g2s(dst + Cfg::RAW_KZ, reinterpret_cast<const uint8_t*>(s.k_sz) + slot * sz, n * sz, full);
          bulk_g2s(dst + Cfg::RAW_IX, static_cast<const uint8_t*>(s.cidx) + slot * id, n * id, full);
          if (ps) bulk_g2s(dst + Cfg::RAW_PS, reinterpret_cast<const uint8_t*>(s.psac) + slot * ps, n * ps, full);
          if (psc) bulk_g2s(dst + Cfg::RAW_PSC, s.psac_scale + slot, n * 2, full);
          bulk_g2s(dst + Cfg::RAW_VC, s.v_code + slot * (D / 16), n * (D / 4), full);
          bulk_g2s(dst + Cfg::RAW_VZ, reinterpret_cast<const uint8_t*>(s.v_sz) + slot * sz, n * sz, full);
        }
        if (out) break;
      }
      // copies still in flight land before the block ends (after an abort the
      // producers no longer wait for them)
      for (int i = max(0, t - Cfg::RS); i < t; ++i)
        mbar_wait(bar + B_RFULL + 8 * (i % Cfg::RS), (i / Cfg::RS) & 1, p.budget);
    }
    }
  } else if (warp >= SW) {
    // ================= producers =================
    set_regs<Cfg::kRegsProd, Cfg::kRegs>();
    // Two threads per key: lanes 8q..8q+7 of a warp take 8 consecutive keys and
    // one half of their channels, so that the 16-byte stores of 8 lanes fall on 8
    // distinct swizzled bank groups.
    const bool values = warp >= Cfg::kValueWarp;
    const int pt = tid - (values ? Cfg::kValueWarp : SW) * 32, pw = pt >> 5;
    const int row = pw * 16 + (lane & 7) + 8 * (lane >> 4), part = (lane >> 3) & 1;
    uint2* frag = reinterpret_cast<uint2*>(smem + Cfg::OFF_FRAG);
    constexpr int QW = N / 16;                    // warps that load query rows
    const int qw = values ? pw : PW + pw;
    static_assert(QW <= 2 * PW, "a warp per 16 query rows");
    int t = 0, seg = 0, frag_src = -1, frag_h = -1;
    // the warp's operand writes are done: one arrival for all lanes
    auto arrive_warp = [&](uint32_t b) __attribute__((always_inline)) {
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(b);
    };

    // The warp has read its part of a packed tile: the stage may be copied over.
    // `seen` is the OR of all that the lane has loaded, so that the arrival waits
    // for the data and not only for the loads' issue: an arrival does not queue
    // behind loads, and while the load/store unit is busy with the rows of the
    // unit before, the next copy could land first. (Without it, 480 units of 120
    // rows and 4 tiles, d = 64: 1,273 of 2,000 calls took a key's coefficients or
    // values from three tiles on.) p.none is 0, which the compiler does not know.
    auto release = [&](uint32_t b, uint32_t seen) __attribute__((always_inline)) {
      const bool read = __all_sync(0xffffffffu, (seen & p.none) == 0u);
      __syncwarp();
      if (read && lane == 0) mbar_arrive(b);
    };

    // The query rows of a unit, a block of 16 rows a warp (of WIDE units by all
    // producers, else by the value warps), which waits for no other: copied raw,
    // 16 bytes a lane and step; their product with the basis (bf16 query, exact; P as two bf16
    // numbers, 2^-16); then both scaled by 2^e per row, max(|q|, |u|) 2^e < 2^15,
    // to fp16.
    auto load_queries = [&]() __attribute__((always_inline)) {
      const RowsSource& s = p.src[w.src];
      constexpr int LPR = D / 8, RPS = 32 / LPR, STEPS = 16 / RPS;      // lanes per row, rows per step, steps per block
      const int c = lane % LPR, r0 = lane / LPR;
      uint8_t* qt = smem + Cfg::OFF_Q;
      float* scr = reinterpret_cast<float*>(smem + Cfg::OFF_SCR) + (seg & 3) * N;
      auto q_off = [&](int rx, int k) { return (rx / kRows) * Cfg::Q_BYTES + int(sw128_off(rx % kRows, k)); };
      // (rows that do not exist are not loaded: their scores are not looked at)
      const int rows = min(N, (w.ql * G - w.rb * N + 15) & ~15);
      const int rb = qw * 16;
      if (seg > 0) mbar_wait_or_abort(bar + B_QEMPTY, (seg - 1) & 1, p.budget, abort);
      if (rb < rows) {
        // lane i finds row i, and the lanes that copy it get its place from there (~0: no such row)
        const int ri = w.rb * N + rb + (lane & 15), i = p.per_head(ri);
        const unsigned long long gr =
            ri < w.ql * G ? ((static_cast<unsigned long long>(w.b) * s.Nq + i) * p.H_q + w.h * G + (ri - i * G)) * D : ~0ull;
#pragma unroll
        for (int st = 0; st < STEPS; ++st) {
          const unsigned long long at = __shfl_sync(0xffffffffu, gr, st * RPS + r0);
          const bool in = at != ~0ull;
          copy16(sb + Cfg::OFF_Q + q_off(rb + st * RPS + r0, c), p.Q + (in ? at : 0) + c * 8, in);
        }
      }
      if (s.r > 0 && (w.src != frag_src || w.h != frag_h)) {
        bar_sync(1, QW * 32);                     // the fragments before are read
        const float* Ph = s.P + size_t(w.h) * D * s.r;
#pragma unroll 1
        for (int i = qw * 32 + lane; i < D / 16 * 2 * 32; i += QW * 32) {
          const int l = i & 31, nt = (i >> 5) & 1, ks = i >> 6;
          const int n = nt * 8 + (l >> 2), k = ks * 16 + 2 * (l & 3);
          float hi[4], lo[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float y = n < s.r ? __ldg(Ph + size_t(k + (e & 1) + 8 * (e >> 1)) * s.r + n) : 0.0f;
            hi[e] = __bfloat162float(__float2bfloat16_rn(y));
            lo[e] = y - hi[e];
          }
          frag[((ks * 2 + nt) * 2 + 0) * 32 + l] = make_uint2(pack_bf16(hi[0], hi[1]), pack_bf16(hi[2], hi[3]));
          frag[((ks * 2 + nt) * 2 + 1) * 32 + l] = make_uint2(pack_bf16(lo[0], lo[1]), pack_bf16(lo[2], lo[3]));
        }
        frag_src = w.src;
        frag_h = w.h;
        bar_sync(1, QW * 32);                     // the fragments are there
      }
      copy_wait();
      __syncwarp();
      if (rb < rows) {
        float acc[2][4], um = 0.0f;               // um: largest |u| of row lane % 16
        if (s.r > 0) {
#pragma unroll
          for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[nt][k] = 0.0f;
#pragma unroll 2
          for (int ks = 0; ks < D / 16; ++ks) {
            uint32_t a[4];
            ldsm_x4(a, sb + Cfg::OFF_Q + q_off(rb + (lane & 15), 2 * ks + (lane >> 4)));
#pragma unroll
            for (int hl = 0; hl < 2; ++hl)
#pragma unroll
              for (int nt = 0; nt < 2; ++nt) {
                const uint2 bb = frag[((ks * 2 + nt) * 2 + hl) * 32 + lane];
                mma16816(acc[nt], a, bb.x, bb.y);
              }
          }
          // rows lane / 4 and lane / 4 + 8
          float u0 = fmaxf(fmaxf(fabsf(acc[0][0]), fabsf(acc[0][1])), fmaxf(fabsf(acc[1][0]), fabsf(acc[1][1])));
          float u1 = fmaxf(fmaxf(fabsf(acc[0][2]), fabsf(acc[0][3])), fmaxf(fabsf(acc[1][2]), fabsf(acc[1][3])));
#pragma unroll
          for (int o = 1; o <= 2; o <<= 1) {
            u0 = fmaxf(u0, __shfl_xor_sync(0xffffffffu, u0, o));
            u1 = fmaxf(u1, __shfl_xor_sync(0xffffffffu, u1, o));
          }
          u0 = __shfl_sync(0xffffffffu, u0, (lane & 7) * 4);
          u1 = __shfl_sync(0xffffffffu, u1, (lane & 7) * 4);
          um = lane & 8 ? u1 : u0;
        }
        // lanes i and i + 16 scale a half of row i each (no lane needs another's
        // row, and eight lanes' chunks fall on eight bank groups)
        const int mine = rb + (lane & 15), k0 = (lane >> 4) * (D / 16);
        __nv_bfloat162 am = __float2bfloat162_rn(0.0f);
#pragma unroll 4
        for (int k = 0; k < D / 16; ++k) {
          const uint4 v = *reinterpret_cast<const uint4*>(qt + q_off(mine, k0 + k));
          const uint32_t u[4] = {v.x & 0x7fff7fffu, v.y & 0x7fff7fffu, v.z & 0x7fff7fffu, v.w & 0x7fff7fffu};
#pragma unroll
          for (int i = 0; i < 4; ++i) am = __hmax2(am, *reinterpret_cast<const __nv_bfloat162*>(&u[i]));
        }
        // (a NaN beside finite values is left out here, and reaches the row's scores through q)
        float top = fmaxf(__low2float(am), __high2float(am));
        top = fmaxf(fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16)), um);
        const int e = top > 0.0f && top < INFINITY ? min(max(15 - exp_above(top), -126), 64) : 0;
        const float qmul = p.q_sign * pow2(e);
#pragma unroll 4
        for (int k = 0; k < D / 16; ++k) {
          uint4* at = reinterpret_cast<uint4*>(qt + q_off(mine, k0 + k));
          const uint4 v = *at;
          const uint32_t u[4] = {v.x, v.y, v.z, v.w};
          uint32_t o4[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            o4[i] = pack_f16(__uint_as_float(u[i] << 16) * qmul, __uint_as_float(u[i] & 0xffff0000u) * qmul);
          *at = make_uint4(o4[0], o4[1], o4[2], o4[3]);
        }
        if (lane < 16) scr[mine] = p.scale_log2 * pow2(-e);
        const int ea = __shfl_sync(0xffffffffu, e, lane >> 2), eb = __shfl_sync(0xffffffffu, e, (lane >> 2) + 8);
        if (s.r > 0) {
          uint8_t* ut = smem + Cfg::OFF_U + (rb / kRows) * Cfg::U_BYTES;
          const int rt = (rb + (lane >> 2)) % kRows, q = (lane & 3) * 4;
          const float ma = p.q_sign * pow2(ea), mb = p.q_sign * pow2(eb);
#pragma unroll
          for (int nt = 0; nt < 2; ++nt) {
            *reinterpret_cast<uint32_t*>(ut + nosw_off(rt, nt) + q) = pack_f16(acc[nt][0] * ma, acc[nt][1] * ma);
            *reinterpret_cast<uint32_t*>(ut + nosw_off(rt + 8, nt) + q) = pack_f16(acc[nt][2] * mb, acc[nt][3] * mb);
          }
        }
      }
      arrive_warp(bar + B_QFULL);
    };

    constexpr int W = CH / 16, Q32 = CH / 32;     // code words, 32-channel runs of a thread
    // byte offset of the scale/zero word of the thread's run q
    auto z_off = [&](int szb, int gshift, int q) __attribute__((always_inline)) {
      return row * szb + ((part * CH + 32 * q) >> gshift) * 4;
    };
    for (; w.more(); w.next(p), ++seg) {
      const RowsSource& s = p.src[w.src];
      const int cnt = w.count(), gshift = s.gshift, szb = (D >> gshift) * 4;
      if (qw < QW) load_queries();
      if (values) {
#pragma unroll 1
        for (int jj = 0; jj < cnt; ++jj, ++t) {
          const bool have = (w.j + jj) * kKeys + row < w.len;
          const int rs = t % Cfg::RS, st = t % VS;
          const uint8_t* raw = smem + Cfg::OFF_RAW + rs * Cfg::RAW_BYTES;
          mbar_wait_or_abort(bar + B_RFULL + 8 * rs, (t / Cfg::RS) & 1, p.budget, abort);
          uint32_t vw[W], vz[Q32];
          load_words<W>(raw + Cfg::RAW_VC + row * (D / 4) + part * (CH / 4), vw);
#pragma unroll
          for (int q = 0; q < Q32; ++q) vz[q] = *reinterpret_cast<const uint32_t*>(raw + Cfg::RAW_VZ + z_off(szb, gshift, q));
          uint32_t seen = 0u;
#pragma unroll
          for (int i = 0; i < W; ++i) seen |= vw[i];
#pragma unroll
          for (int q = 0; q < Q32; ++q) seen |= vz[q];
          release(bar + B_REMPTY + 8 * rs, seen);
          if (!have) {                            // a code of zero, scale and zero of zero
#pragma unroll
            for (int q = 0; q < Q32; ++q) vz[q] = 0u;
          }
          if (t >= VS) mbar_wait_or_abort(bar + B_VEMPTY + 8 * st, (t / VS - 1) & 1, p.budget, abort);
          uint8_t* vt = smem + Cfg::OFF_V + st * Cfg::V_BYTES;
#pragma unroll
          for (int q = 0; q < Q32; ++q) {
            const uint32_t s2 = __byte_perm(vz[q], 0u, 0x1010u), z2 = __byte_perm(vz[q], 0u, 0x3232u);
            const uint32_t add[4] = {z2, z2, z2, z2};
#pragma unroll
            for (int c = 0; c < 4; ++c)
              *reinterpret_cast<uint4*>(vt + sw128_off(row, part * (CH / 8) + 4 * q + c)) =
                  dequant8(vw[2 * q + (c >> 1)], c, s2, add);
          }
          arrive_warp(bar + B_VFULL + 8 * st);
        }
      } else {
        const uint4* cent4 = reinterpret_cast<const uint4*>(s.cent) + size_t(w.h) * s.M * (D / 8) + part * (CH / 8);
        const int r = s.r, top = s.M - 1;
        const bool int8 = s.psac_fmt == 1, wide = s.M > 256;
        constexpr int CP = 8;              // PSAC coefficients of a thread
#pragma unroll 1
        for (int jj = 0; jj < cnt; ++jj, ++t) {
          const bool have = (w.j + jj) * kKeys + row < w.len;
          const int rs = t % Cfg::RS, st = t % KS;
          const uint8_t* raw = smem + Cfg::OFF_RAW + rs * Cfg::RAW_BYTES;
          mbar_wait_or_abort(bar + B_RFULL + 8 * rs, (t / Cfg::RS) & 1, p.budget, abort);
          const int id = wide ? reinterpret_cast<const uint16_t*>(raw + Cfg::RAW_IX)[row] : raw[Cfg::RAW_IX + row];
          // (an id is only followed where the token exists)
          const uint4* m4 = cent4 + size_t(have ? min(id, top) : 0) * (D / 8);
          uint4 mu[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) mu[c] = __ldg(m4 + c);
          uint32_t kw[W], kz[Q32], ps[CP / 2];
          load_words<W>(raw + row * (D / 4) + part * (CH / 4), kw);
#pragma unroll
          for (int q = 0; q < Q32; ++q) kz[q] = *reinterpret_cast<const uint32_t*>(raw + Cfg::RAW_KZ + z_off(szb, gshift, q));
#pragma unroll
          for (int i = 0; i < CP / 2; ++i) ps[i] = 0u;
          if (have) {
            if (int8) {
              // fp16(code * the token's scale)
              const float sc = __half2float(reinterpret_cast<const __half*>(raw + Cfg::RAW_PSC)[row]);
#pragma unroll
              for (int e = 0; e < CP; e += 8) {
                if (part * CP + e < r) {
                  const uint2 two = *reinterpret_cast<const uint2*>(raw + Cfg::RAW_PS + row * r + part * CP + e);
#pragma unroll
                  for (int i = 0; i < 4; ++i) {
                    const uint32_t q = ((i < 2 ? two.x : two.y) >> (16 * (i & 1))) & 0xffffu;
                    ps[e / 2 + i] = pack_f16(float(int8_t(q & 0xff)) * sc, float(int8_t(q >> 8)) * sc);
                  }
                }
              }
            } else {
#pragma unroll
              for (int e = 0; e < CP; e += 8)
                if (part * CP + e < r) load_words<4>(raw + Cfg::RAW_PS + (row * r + part * CP + e) * 2, ps + e / 2);
            }
          }
          uint32_t seen = uint32_t(id);
#pragma unroll
          for (int i = 0; i < W; ++i) seen |= kw[i];
#pragma unroll
          for (int q = 0; q < Q32; ++q) seen |= kz[q];
#pragma unroll
          for (int i = 0; i < CP / 2; ++i) seen |= ps[i];
          release(bar + B_REMPTY + 8 * rs, seen);
          if (!have) {                            // codes, scale, zero and centre of zero
#pragma unroll
            for (int q = 0; q < Q32; ++q) kz[q] = 0u;
          }
          if (t >= KS) mbar_wait_or_abort(bar + B_KEMPTY + 8 * st, (t / KS - 1) & 1, p.budget, abort);
          uint8_t* kt = smem + Cfg::OFF_K + st * Cfg::K_BYTES;
#pragma unroll
          for (int q = 0; q < Q32; ++q) {
            uint4 next[4];
            if (q + 1 < Q32) {
#pragma unroll
              for (int c = 0; c < 4; ++c) next[c] = __ldg(m4 + 4 * (q + 1) + c);
            }
            const uint32_t s2 = __byte_perm(kz[q], 0u, 0x1010u), z2 = __byte_perm(kz[q], 0u, 0x3232u);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const uint4 m = have ? mu[c] : make_uint4(0, 0, 0, 0);
              const uint32_t add[4] = {hadd2(z2, m.x), hadd2(z2, m.y), hadd2(z2, m.z), hadd2(z2, m.w)};
              *reinterpret_cast<uint4*>(kt + sw128_off(row, part * (CH / 8) + 4 * q + c)) =
                  dequant8(kw[2 * q + (c >> 1)], c, s2, add);
            }
            if (q + 1 < Q32) {
#pragma unroll
              for (int c = 0; c < 4; ++c) mu[c] = next[c];
            }
          }
          uint8_t* at = smem + Cfg::OFF_A + st * Cfg::A_BYTES;
#pragma unroll
          for (int e = 0; e < CP; e += 8)
            *reinterpret_cast<uint4*>(at + nosw_off(row, (part * CP + e) / 8)) =
                make_uint4(ps[e / 2], ps[e / 2 + 1], ps[e / 2 + 2], ps[e / 2 + 3]);
          arrive_warp(bar + B_KFULL + 8 * st);
        }
      }
    }
  } else {
    // ================= softmax (thread = row = TMEM lane) =================
    set_regs<Cfg::kRegsSoft, Cfg::kRegs>();
    const int x = warp >> 2, wq = warp & 3, row = wq * 32 + lane, ru = (WIDE ? x * kRows : 0) + row;
    const uint32_t lane_base = uint32_t(wq * 32) << 16;
    const uint32_t tS = tmem + x * kKeys + lane_base, tO = tmem + 2 * kKeys + x * kRows + lane_base;
    float2* ml_s = reinterpret_cast<float2*>(smem + Cfg::OFF_ML);
    // a wait of the lane ran out, or before the last vote one of the warp (below, of both groups)
    bool dead = false;
    int t0 = 0, seg = 0, k = 0;                   // the part's first tile; tiles of this group
    for (; w.more(); w.next(p), ++seg) {
      const RowsSource& s = p.src[w.src];
      const int cnt = w.count(), j0 = w.j, len = w.len;
      const int live = w.ql * G - w.rb * N;       // rows of the unit
      const bool row_ok = ru < live, warp_ok = ru - lane < live;
      const int jx = WIDE ? 0 : (x - t0) & 1;     // the group's first tile of the part
      // (a row whose first scores are not numbers does not move m: its p are NaN by nm)
      float m = -INFINITY, l = 0.0f, base = 0.0f, sc = 0.0f, nm = __int_as_float(0x7fc00000);
      for (int jj = jx; jj < cnt; jj += WIDE ? 1 : 2, ++k) {
        dead |= !mbar_wait_or_abort(bar + B_SFULL + 8 * x, k & 1, p.budget, abort);
        fence_after_sync();
        if (warp_ok) {
          const bool first = jj == jx;
          if (first) base = reinterpret_cast<const float*>(smem + Cfg::OFF_SCR)[(seg & 3) * N + ru];
          const int lim = len - (j0 + jj) * kKeys;             // keys of the tile
          const bool full = lim >= kKeys;
          // the tile's maximum, 8 independent chains
          float mp[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) mp[i] = -INFINITY;
#pragma unroll 1
          for (int c0 = 0; c0 < kKeys; c0 += 32) {
            uint32_t r[32];
            tmem_ld32_issue(tS + c0, r);
            tmem_wait_ld(r);
            if (full) {
#pragma unroll
              for (int i = 0; i < 32; i += 2)
                mp[(i >> 1) & 7] = fmax3(mp[(i >> 1) & 7], __uint_as_float(r[i]), __uint_as_float(r[i + 1]));
            } else {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (c0 + i < lim) mp[i & 7] = fmaxf(mp[i & 7], __uint_as_float(r[i]));
            }
          }
          const float tm = base * fmaxf(fmaxf(fmaxf(mp[0], mp[1]), fmaxf(mp[2], mp[3])),
                                        fmaxf(fmaxf(mp[4], mp[5]), fmaxf(mp[6], mp[7])));
          const bool up = tm > m + kTrail;
          if (__any_sync(0xffffffffu, up)) {
            // a row's maximum moves up: its sums follow (by an exact power of two)
            const float mn = up ? ceilf(tm) : m;
            const float alpha = up ? ex2(m - mn) : 1.0f;       // (m = -inf: 0, nothing summed yet)
            m = mn;
            l *= alpha;
            if (up) {
              // s sc - m is one fma, exact to half a step of m: beyond 2^20 (where a
              // key's fp16 rounding already moves the score by 2^8) the row's scores
              // are taken at a 2^-i of their size, so that this stays small
              const float damp =
                  fabsf(mn) > 0x1p20f && fabsf(mn) < INFINITY ? pow2(-max(exp_above(fabsf(mn)) - 21, 0)) : 1.0f;
              sc = base * damp;
              nm = kBias - mn * damp;
            }
            if (!first) {                         // (the scores came after P . V of the group's tile before)
#pragma unroll 1
              for (int c0 = 0; c0 < D; c0 += 32) {
                uint32_t r[32];
                float v[32];
                tmem_ld32_issue(tO + c0, r);
                tmem_wait_ld(r);
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]) * alpha;
                tmem_st32(tO + c0, v);
              }
            }
          }
          const f32x2 sc2 = pk2(sc, sc), nm2 = pk2(nm, nm);
          f32x2 sum[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll 1
          for (int c0 = 0; c0 < kKeys; c0 += 32) {
            uint32_t r[32], pw[16];
            tmem_ld32_issue(tS + c0, r);
            tmem_wait_ld(r);
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const float2 y = up2(ffma2(pk2(__uint_as_float(r[i]), __uint_as_float(r[i + 1])), sc2, nm2));
              float p0 = ex2(y.x), p1 = ex2(y.y);
              if (!full) {
                p0 = c0 + i < lim ? p0 : 0.0f;
                p1 = c0 + i + 1 < lim ? p1 : 0.0f;
              }
              sum[(i >> 1) & 3] = fadd2(sum[(i >> 1) & 3], pk2(p0, p1));
              pw[i / 2] = pack_f16(p0, p1);
            }
            tmem_st16(tS + c0 / 2, pw);           // over columns already read
          }
          tmem_wait_st();
          const float2 s01 = up2(fadd2(sum[0], sum[1])), s23 = up2(fadd2(sum[2], sum[3]));
          l += (s01.x + s23.x) + (s01.y + s23.y);
        }
        fence_before_sync();
        // (the lanes of a wait that failed have spoilt rows of this warp alone)
        dead = __any_sync(0xffffffffu, dead);
        if (dead) break;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar + B_PFULL + 8 * x);
      }
      // ---- the unit's rows: a group's 128 rows, or half their channels of both groups' sums
      if (jx < cnt && !dead) dead = !mbar_wait_or_abort(bar + B_PDONE + 8 * x, (k - 1) & 1, p.budget, abort);
      dead = __any_sync(0xffffffffu, dead || *abort);
      fence_after_sync();
      float f0 = 1.0f, f1 = 0.0f;
      if constexpr (!WIDE) {
        ml_s[x * kRows + row] = make_float2(m, l);
        dead = bar_or(2, 256, dead);
        fence_after_sync();                       // the other group's sums too
        const float2 a = ml_s[row], b = ml_s[kRows + row];
        m = fmaxf(a.y == 0.0f ? -INFINITY : a.x, b.y == 0.0f ? -INFINITY : b.x);
        f0 = a.y == 0.0f ? 0.0f : ex2(a.x - m);
        f1 = b.y == 0.0f ? 0.0f : ex2(b.x - m);
        l = f0 * a.y + f1 * b.y;
      }
      const bool whole = j0 == 0 && cnt == tiles_of(len);
      if (dead) {
        // (a sum that is not a number reaches the merged row whatever the weight of
        // its piece; channels alone are not looked at where the weight is 0)
        m = 0.0f;
        l = __int_as_float(0x7fc00000);
      }
      if (warp_ok) {
        const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
        const int ri = w.rb * N + ru, i = p.per_head(ri);
        const size_t gr = (size_t(w.b) * s.Nq + i) * p.H_q + w.h * G + (ri - i * G);
        const size_t pr = (size_t(blockIdx.x) * 2 + (j0 > 0 ? 0 : 1)) * N + ru;
        float* po = !whole ? p.part_o + pr * D : p.dir_o + (size_t(w.src) * p.dir_rows + gr) * D;
        if (row_ok && (WIDE || x == 0)) {
          // (sums carry 2^kBias: the stored maximum takes it out)
          if (!whole) p.part_ml[pr] = make_float2(m - kBias, l);
          else if (!p.out) p.dir_ml[size_t(w.src) * p.dir_rows + gr] = make_float2(m - kBias, l);
        }
        const int c_lo = WIDE ? 0 : x * (D / 2), c_hi = WIDE ? D : c_lo + D / 2;
        const bool has0 = !WIDE && (cnt > 1 || (t0 & 1) == 0), has1 = !WIDE && (cnt > 1 || (t0 & 1) == 1);
#pragma unroll 1
        for (int c0 = c_lo; c0 < c_hi; c0 += 32) {
          float v[32];
          uint32_t r[32];
          if constexpr (WIDE) {
            tmem_ld32_issue(tO + c0, r);          // every lane: warp-wide TMEM load
            tmem_wait_ld(r);
#pragma unroll
            for (int q = 0; q < 32; ++q) v[q] = __uint_as_float(r[q]);
          } else {
            const uint32_t tB = tmem + 2 * kKeys + lane_base + c0;
#pragma unroll
            for (int q = 0; q < 32; ++q) v[q] = 0.0f;
            if (has0) {
              tmem_ld32_issue(tB, r);
              tmem_wait_ld(r);
              if (f0 != 0.0f) {
#pragma unroll
                for (int q = 0; q < 32; ++q) v[q] = f0 * __uint_as_float(r[q]);
              }
            }
            if (has1) {
              tmem_ld32_issue(tB + kRows, r);
              tmem_wait_ld(r);
              if (f1 != 0.0f) {
#pragma unroll
                for (int q = 0; q < 32; ++q) v[q] = fmaf(f1, __uint_as_float(r[q]), v[q]);
              }
            }
          }
          if (dead) {
#pragma unroll
            for (int q = 0; q < 32; ++q) v[q] = __int_as_float(0x7fc00000);
          }
          if constexpr (WIDE) {
            // 64 bytes a row (16 fp32 or 32 bf16 channels) through shared memory, so that
            // four lanes write a row's: a row a lane would take 32 lines a store, and the
            // load/store unit that the next unit's queries pass through
            const bool f32 = !whole || !p.out || p.out_dtype == KV2_OUT_F32;
            const float mul = whole && p.out ? inv : 1.0f;
            uint8_t* stg = smem + Cfg::OFF_STG + warp * 2048;
            const unsigned long long mine =
                !row_ok ? 0ull
                : !whole || !p.out ? reinterpret_cast<unsigned long long>(po + c0)
                                   : reinterpret_cast<unsigned long long>(p.out) + (gr * D + c0) * (f32 ? 4 : 2);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              if (half && !f32) break;
              uint4 o4[4];
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                if (f32) {
                  const float* f = v + 16 * half + 4 * q;
                  o4[q] = make_uint4(__float_as_uint(f[0] * mul), __float_as_uint(f[1] * mul), __float_as_uint(f[2] * mul), __float_as_uint(f[3] * mul));
                } else {
                  const float* f = v + 8 * q;
                  o4[q] = make_uint4(pack_bf16(f[0] * mul, f[1] * mul), pack_bf16(f[2] * mul, f[3] * mul),
                                     pack_bf16(f[4] * mul, f[5] * mul), pack_bf16(f[6] * mul, f[7] * mul));
                }
              }
              __syncwarp();                       // the rows before are read
#pragma unroll
              for (int q = 0; q < 4; ++q) *reinterpret_cast<uint4*>(stg + lane * 64 + ((q ^ (lane >> 1)) & 3) * 16) = o4[q];
              __syncwarp();
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int rr = i * 8 + (lane >> 2);
                const unsigned long long to = __shfl_sync(0xffffffffu, mine, rr);
                const uint4 x = *reinterpret_cast<const uint4*>(stg + rr * 64 + (((lane & 3) ^ (rr >> 1)) & 3) * 16);
                if (to) *reinterpret_cast<uint4*>(to + half * 64 + (lane & 3) * 16) = x;
              }
            }
            continue;
          }
          if (!row_ok) continue;
          if (!whole || !p.out) {
            float4* dst = reinterpret_cast<float4*>(po + c0);
#pragma unroll
            for (int q = 0; q < 32; q += 4) dst[q / 4] = make_float4(v[q], v[q + 1], v[q + 2], v[q + 3]);
          } else if (p.out_dtype == KV2_OUT_F32) {
            float4* dst = reinterpret_cast<float4*>(static_cast<float*>(p.out) + gr * D + c0);
#pragma unroll
            for (int q = 0; q < 32; q += 4) dst[q / 4] = make_float4(v[q] * inv, v[q + 1] * inv, v[q + 2] * inv, v[q + 3] * inv);
          } else {
            uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + gr * D + c0);
#pragma unroll
            for (int q = 0; q < 32; q += 8)
              dst[q / 8] = make_uint4(pack_bf16(v[q] * inv, v[q + 1] * inv), pack_bf16(v[q + 2] * inv, v[q + 3] * inv),
                                      pack_bf16(v[q + 4] * inv, v[q + 5] * inv), pack_bf16(v[q + 6] * inv, v[q + 7] * inv));
          }
        }
      }
      // both groups' sums are read before the next unit's P . V starts them afresh
      if constexpr (!WIDE) bar_sync(2, 256);
      t0 += cnt;
    }
  }

  // the merge (this grid's programmatic dependent) may be scheduled; it waits
  // for this grid before it reads anything, and so, through this wait, for the
  // split decode kernel that this grid may have been launched beside
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  fence_before_sync();
  __syncthreads();
  if (warp == Cfg::kMmaWarp) {
    if (*abort) {
      if (elect_one()) {                          // (the lane that issued the MMAs)
        atomicExch(p.err, 1);
        mma_commit(bar + B_FINAL);                // wait (bounded) for MMAs in flight
      }
      __syncwarp();
      mbar_wait(bar + B_FINAL, 0, 1ull << 32);
    }
    fence_after_sync();
    tmem_dealloc(tmem, Cfg::kTmemCols);
  }
}

// ---------------------------------------------------------------------------
// merges
// ---------------------------------------------------------------------------

// A lane's W = D / 32 channels of a row: W * lane ...
template <int W>
struct RowPart {
  float v[W];
  __device__ __forceinline__ static RowPart load(const float* row, int lane) {
    RowPart r;
#pragma unroll
    for (int i = 0; i < W; i += 2) {              // (the split decode kernel's rows start on 8 bytes)
      const float2 x = *reinterpret_cast<const float2*>(row + W * lane + i);
      r.v[i] = x.x; r.v[i + 1] = x.y;
    }
    return r;
  }
  // += f * o, o not looked at where f is 0 (an empty or absent piece)
  __device__ __forceinline__ void add(float f, const RowPart& o) {
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = f == 0.0f ? v[i] : fmaf(f, o.v[i], v[i]);
  }
  // the row of the output, divided by its sum l (0: an empty row)
  __device__ __forceinline__ void store(void* out, int out_dtype, size_t row, int lane, float l) const {
    const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
    float* f = static_cast<float*>(out) + row * (W * 32) + W * lane;
    __nv_bfloat16* b = static_cast<__nv_bfloat16*>(out) + row * (W * 32) + W * lane;
    if (out_dtype == KV2_OUT_F32) {
      if constexpr (W == 4) *reinterpret_cast<float4*>(f) = make_float4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
      else *reinterpret_cast<float2*>(f) = make_float2(v[0] * inv, v[1] * inv);
    } else {
      if constexpr (W == 4) *reinterpret_cast<uint2*>(b) = make_uint2(pack_bf16(v[0] * inv, v[1] * inv), pack_bf16(v[2] * inv, v[3] * inv));
      else *reinterpret_cast<uint32_t*>(b) = pack_bf16(v[0] * inv, v[1] * inv);
    }
  }
};

// One warp: log-sum-exp of n partial results of a row; ml(i) is the maximum
// and the sum of part i (sum 0: an empty part), o(i) its row of channels.
template <int W, class ML, class O>
__device__ __forceinline__ void merge_parts(int n, int lane, ML ml, O o, float& m, float& l, RowPart<W>& acc) {
  m = -INFINITY;
  for (int i = lane; i < n; i += 32) {
    const float2 x = ml(i);
    if (!(x.y == 0.0f)) m = fmaxf(m, x.x);
  }
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
  l = 0.0f;
#pragma unroll
  for (int i = 0; i < W; ++i) acc.v[i] = 0.0f;
  for (int i0 = 0; i0 < n; i0 += 32) {
    float f = 0.0f;
    if (i0 + lane < n) {
      const float2 x = ml(i0 + lane);
      if (!(x.y == 0.0f)) {
        f = exp2f(x.x - m);
        l = fmaf(f, x.y, l);
      }
    }
    // eight rows in flight together
    const int end = min(32, n - i0);
    for (int k = 0; k < end; k += 8) {
      RowPart<W> x[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (k + u < end) x[u] = RowPart<W>::load(o(i0 + k + u), lane);
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const float fk = __shfl_sync(0xffffffffu, f, (k + u) & 31);
        if (k + u < end) acc.add(fk, x[u]);
      }
    }
  }
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) l += __shfl_xor_sync(0xffffffffu, l, k);
}
// the pieces of CTAs c0 (slot 1) and c0 + 1 .. c1 (slot 0); T >= C or a part may be empty
template <int D>
__device__ __forceinline__ void merge_pieces(const RowsParams& p, int N, int row, int c0, int c1, long long T, int C,
                                            int lane, float& m, float& l, RowPart<D / 32>& o) {
  auto at = [&](int i) { return (size_t(c0 + i) * 2 + (i == 0)) * N + row; };
  merge_parts<D / 32>(
      c1 - c0 + 1, lane,
      [&](int i) { return T >= C || part_begin(T, c0 + i, C) < part_begin(T, c0 + i + 1, C) ? p.part_ml[at(i)] : make_float2(0.0f, 0.0f); },
      [&](int i) { return p.part_o + at(i) * D; }, m, l, o);
}

// One source: blocks (c - 1, .) merge the unit that the border before CTA c
// cuts, kCutRows rows a block; the blocks of a unit's K borders share its rows
// (with parts that are empty, T < C, the first border has them all). The way
// to the rows (list, lengths, borders) is a chain of reads, so a warp takes
// several rows, and where a unit has just two pieces, as most do with many
// query rows, all their reads go out together. Cross attention of 4 x 509
// queries over 2,047 keys and 32 heads: 11 us for 26.7 us with one row a warp.
constexpr int kCutRows = 64;
template <int D, int N>
__global__ void __launch_bounds__(256) rows_merge_cut(const __grid_constant__ RowsParams p, int C) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int W = D / 32, R = kCutRows / 8;
  const int c = blockIdx.x + 1, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int4 at = p.cta[c];
  const long long T = *p.total, lo = part_begin(T, c, C);
  if (lo >= part_begin(T, c + 1, C)) return;
  if (at.w == 0) return;                          // no unit is cut here
  const int G = p.H_q / p.H_kv;
  const int ql = seq_queries(p.src[0], at.y), RB = blocks_of<N>(ql, G);
  const long long u = lo - at.w;                  // position of the unit's first tile
  const int c0 = part_of(u, T, C), c1 = part_of(u + tiles_of(seq_len(p.src[0], at.y)) - 1, T, C);
  const int K = T < C ? 1 : c1 - c0, k = T < C ? 0 : c - 1 - c0;
  if (T < C && part_begin(T, c0 + 1, C) != lo) return;
  const int first = blockIdx.y * kCutRows + warp * R, base = (at.z % RB) * N, h = at.z / RB;
  auto out_row = [&](int row) {
    const int ri = base + row, i = p.per_head(ri);
    return (size_t(at.y) * p.src[0].Nq + i) * p.H_q + h * G + (ri - i * G);
  };
  const int rows = min(R, ql * G - base - first);
  if (c1 == c0 + 1) {
    const size_t a0 = (size_t(c0) * 2 + 1) * N + first, a1 = size_t(c1) * 2 * N + first;
#pragma unroll
    for (int i0 = 0; i0 < R; i0 += 4) {
      RowPart<W> x[4], y[4];
      float2 mx[4], my[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i0 + i >= rows) break;
        mx[i] = p.part_ml[a0 + i0 + i];
        my[i] = p.part_ml[a1 + i0 + i];
        x[i] = RowPart<W>::load(p.part_o + (a0 + i0 + i) * D, lane);
        y[i] = RowPart<W>::load(p.part_o + (a1 + i0 + i) * D, lane);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i0 + i >= rows) break;
        const bool ex = mx[i].y == 0.0f, ey = my[i].y == 0.0f;
        const float m = fmaxf(ex ? -INFINITY : mx[i].x, ey ? -INFINITY : my[i].x);
        const float fx = ex ? 0.0f : exp2f(mx[i].x - m), fy = ey ? 0.0f : exp2f(my[i].x - m);
        RowPart<W> o{};
        o.add(fx, x[i]);
        o.add(fy, y[i]);
        o.store(p.out, p.out_dtype, out_row(first + i0 + i), lane, fmaf(fx, mx[i].y, fy * my[i].y));
      }
    }
    return;
  }
#pragma unroll 1
  for (int i = (k + K - first % K) % K; i < rows; i += K) {   // the unit's rows k, k + K, ...
    float m, l;
    RowPart<W> o;
    merge_pieces<D>(p, N, first + i, c0, c1, T, C, lane, m, l, o);
    o.store(p.out, p.out_dtype, out_row(first + i), lane, l);
  }
}

// Shared prefix: one warp per (sequence, query head) joins the row's result
// over the prefix and over the sequence's own cache, each whole or in pieces.
template <int D, int N>
__global__ void __launch_bounds__(256) rows_merge_shared(const __grid_constant__ RowsParams p, int C) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long gr = static_cast<long long>(blockIdx.x) * 8 + warp;
  if (gr >= p.dir_rows) return;
  const int G = p.H_q / p.H_kv, hq = int(gr % p.H_q), h = hq / G, g = hq % G;
  const long long T = *p.total;
  float m[2], l[2];
  RowPart<D / 32> o[2];
  if (p.split_part) {
    // own cache: the splits' rows [G][D + 2], maximum and sum behind the channels
    const float* base = p.split_part + (gr / p.H_q * p.H_kv + h) * size_t(p.splits) * G * (D + 2) + size_t(g) * (D + 2);
    const size_t step = size_t(G) * (D + 2);
    merge_parts<D / 32>(
        p.splits, lane, [&](int i) { return *reinterpret_cast<const float2*>(base + i * step + D); },
        [&](int i) { return base + i * step; }, m[1], l[1], o[1]);
  }
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    if (s == 1 && p.split_part) break;
    const RowsSource& src = p.src[s];
    const int seq = int(gr / p.H_q), b = seq / src.Nq, i = seq % src.Nq;
    const int nb = tiles_of(seq_len(src, b)), RB = blocks_of<N>(src.Nq, G);
    const int ri = i * G + g;
    const long long u = p.base[(s ? p.src[0].B : 0) + b] +
                        (static_cast<long long>(h) * RB + ri / N) * (nb + kLead) + kLead;
    const int c0 = part_of(u, T, C), c1 = part_of(u + nb - 1, T, C);
    if (c0 == c1) {
      const float2 ml = p.dir_ml[size_t(s) * p.dir_rows + gr];
      m[s] = ml.x;
      l[s] = ml.y;
      o[s] = RowPart<D / 32>::load(p.dir_o + (size_t(s) * p.dir_rows + gr) * D, lane);
    } else {
      merge_pieces<D>(p, N, ri % N, c0, c1, T, C, lane, m[s], l[s], o[s]);
    }
  }
  const float mm = fmaxf(l[0] == 0.0f ? -INFINITY : m[0], l[1] == 0.0f ? -INFINITY : m[1]);
  const float f0 = l[0] == 0.0f ? 0.0f : exp2f(m[0] - mm), f1 = l[1] == 0.0f ? 0.0f : exp2f(m[1] - mm);
  RowPart<D / 32> r{};
  r.add(f0, o[0]);
  r.add(f1, o[1]);
  r.store(p.out, p.out_dtype, size_t(gr), lane, f0 * l[0] + f1 * l[1]);
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------

int sm_count() {
  int dev = 0, n = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  return n > 0 ? n : 148;
}

// rows per unit for the most rows that read the same keys
int unit_rows(long long rows) { return rows <= kRows ? kRows : 2 * kRows; }

// workspace: header (word 0 the error word, the tile count at byte 16), the
// first tile of every sequence, the CTAs' places, pieces, whole units
struct RowsPlan {
  int N, C, listed, splits;   // sources in the work list; splits of the own caches by the decode kernel (0: listed)
  long long rows;
  size_t base, cta, part_ml, part_o, dir_ml, dir_o, split, bytes;
};
size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

RowsPlan plan_rows(const RowsArgs& a) {
  RowsPlan pl{};
  const int G = a.H_q / a.src[0].c->H_kv, d = a.src[0].c->d;
  // The sequences' own caches have G rows a unit. With more such units than SMs
  // the split decode kernel, where it is built for them, takes them sooner (64
  // sequences x 8 heads of up to 515 tokens behind a 32,768-token prefix: 133 us
  // against 200 us); with fewer its launch costs more than they do in the list
  // (8 x 8 of up to 256: 82 against 75 us).
  const bool by_decode = a.nsrc == 2 && (G == 1 || G == 2 || G == 4 || G == 8) &&
                         static_cast<long long>(a.src[1].c->B) * a.src[1].c->H_kv > sm_count();
  pl.listed = by_decode ? 1 : a.nsrc;
  if (pl.listed < a.nsrc) pl.splits = decode_splits(*a.src[1].c, a.H_q, a.src[1].max_len);
  long long most = 0;
  for (int s = 0; s < pl.listed; ++s) most = std::max(most, static_cast<long long>(a.src[s].Nq) * G);
  pl.N = unit_rows(most);
  long long tiles = 0;
  size_t seqs = 0;
  for (int s = 0; s < pl.listed; ++s) {
    const long long rows = static_cast<long long>(a.src[s].Nq) * G;
    tiles += static_cast<long long>(std::max(1, (a.src[s].max_len + kKeys - 1) / kKeys)) * ((rows + pl.N - 1) / pl.N) *
             a.src[s].c->H_kv * a.src[s].c->B;
    seqs += size_t(a.src[s].c->B);
  }
  pl.C = int(std::min<long long>(sm_count(), std::max<long long>(tiles, 1)));
  pl.rows = static_cast<long long>(a.src[0].c->B) * a.src[0].Nq * a.H_q;
  pl.base = 256;
  pl.cta = pl.base + up256(seqs * 8);
  pl.part_ml = pl.cta + up256(size_t(pl.C) * 16);
  pl.part_o = pl.part_ml + up256(size_t(pl.C) * 2 * pl.N * 8);
  pl.dir_ml = pl.part_o + up256(size_t(pl.C) * 2 * pl.N * d * 4);
  pl.dir_o = pl.dir_ml + (a.nsrc == 2 ? up256(size_t(pl.listed) * pl.rows * 8) : 0);
  pl.split = pl.dir_o + (a.nsrc == 2 ? up256(size_t(pl.listed) * pl.rows * d * 4) : 0);
  pl.bytes = pl.split + size_t(a.src[0].c->H_kv) * (a.nsrc == 2 ? a.src[1].c->B : 0) * pl.splits * G * (d + 2) * 4;
  return pl;
}

template <int D, bool WIDE>
cudaError_t launch_cfg(const RowsParams& p, const RowsPlan& pl, cudaStream_t s) {
  using Cfg = RCfg<D, WIDE>;
  auto kern = rows_attn_kernel<D, WIDE>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(Cfg::SMEM));
  if (e != cudaSuccess) return e;
  // the role split spends exactly these registers: with fewer at launch it would wait for ever
  cudaFuncAttributes fa;
  e = cudaFuncGetAttributes(&fa, kern);
  if (e != cudaSuccess) return e;
  if (fa.numRegs != Cfg::kRegs) return cudaErrorInvalidConfiguration;
  const bool both = p.dir_o != nullptr;       // a shared prefix: rows are joined by the merge
  RowsParams q = p;
  if (both) q.out = nullptr;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(pl.C);
  cfg.blockDim = dim3(Cfg::kThreads);
  cfg.dynamicSmemBytes = Cfg::SMEM;
  cfg.stream = s;
  if (pl.splits) {                            // beside the last blocks of the split decode kernel
    cfg.attrs = attr;
    cfg.numAttrs = 1;
  }
  e = cudaLaunchKernelEx(&cfg, kern, q);
  if (e != cudaSuccess || (!both && pl.C == 1)) return e;
  cfg = cudaLaunchConfig_t{};
  cfg.gridDim = both ? dim3(unsigned((pl.rows + 7) / 8)) : dim3(pl.C - 1, Cfg::N / kCutRows);
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, both ? rows_merge_shared<D, Cfg::N> : rows_merge_cut<D, Cfg::N>, p, pl.C);
}

template <int D>
cudaError_t launch_d(const RowsParams& p, const RowsPlan& pl, cudaStream_t s) {
  return pl.N == kRows ? launch_cfg<D, false>(p, pl, s) : launch_cfg<D, true>(p, pl, s);
}

}  // namespace

size_t rows_workspace_bytes(const RowsArgs& a) { return plan_rows(a).bytes; }

cudaError_t launch_rows(const RowsArgs& a, cudaStream_t s) {
  const RowsPlan pl = plan_rows(a);
  if (pl.rows == 0) return cudaSuccess;
  RowsParams p{};
  for (int i = 0; i < a.nsrc; ++i) {
    const kv2_cache& c = *a.src[i].c;
    RowsSource& q = p.src[i];
    q.k_code = c.k_code; q.v_code = c.v_code; q.k_sz = c.k_sz; q.v_sz = c.v_sz;
    q.cidx = c.cidx; q.psac = c.psac; q.psac_scale = c.psac_scale; q.cent = c.centroids; q.P = c.P;
    q.table = c.block_table;
    q.lens = a.src[i].lens;
    q.q_lens = a.src[i].q_lens;
    q.B = c.B; q.M = c.M; q.r = c.r; q.cap = c.capacity; q.page = c.page_tokens; q.psac_fmt = c.psac_fmt;
    const int group = cache_group(c);
    q.gshift = group == 128 ? 7 : group == 64 ? 6 : 5;
    q.max_len = a.src[i].max_len;
    q.Nq = a.src[i].Nq;
  }
  char* ws = static_cast<char*>(a.ws);
  p.nsrc = pl.listed;
  p.H_kv = a.src[0].c->H_kv;
  p.H_q = a.H_q;
  p.by_group = row_division(uint32_t(a.H_q / p.H_kv));
  p.Q = a.Q;
  p.out = a.out;
  p.out_dtype = a.out_dtype;
  p.scale_log2 = fabsf(a.sm_scale) * 1.4426950408889634f;
  p.q_sign = a.sm_scale < 0.0f ? -1.0f : 1.0f;
  p.none = 0u;
  p.err = reinterpret_cast<int*>(ws);
  p.total = reinterpret_cast<long long*>(ws + 16);
  p.base = reinterpret_cast<long long*>(ws + pl.base);
  p.cta = reinterpret_cast<int4*>(ws + pl.cta);
  p.part_ml = reinterpret_cast<float2*>(ws + pl.part_ml);
  p.part_o = reinterpret_cast<float*>(ws + pl.part_o);
  p.dir_ml = reinterpret_cast<float2*>(ws + pl.dir_ml);
  p.dir_o = a.nsrc == 2 ? reinterpret_cast<float*>(ws + pl.dir_o) : nullptr;
  p.dir_rows = pl.rows;
  if (pl.splits) {
    float* part = reinterpret_cast<float*>(ws + pl.split);
    DecodeArgs d{a.src[1].c, a.src[1].max_len, a.H_q, a.Q, a.sm_scale, nullptr, a.out_dtype, a.ws, 0};
    d.rows = true;
    d.lens = a.src[1].lens;
    p.split_part = part;
    p.splits = pl.splits;
    const cudaError_t e = launch_decode_split(d, part, s);
    if (e != cudaSuccess) return e;
  }
  p.force_timeout = env_force_timeout_ctas();
  p.budget = p.force_timeout == 1 ? (1ull << 20) : env_wait_budget();
  return a.src[0].c->d == 64 ? launch_d<64>(p, pl, s) : launch_d<128>(p, pl, s);
}

}  // namespace kv2
