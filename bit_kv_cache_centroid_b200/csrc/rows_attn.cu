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
// Both products are computed transposed, keys (then channels) in the 128 rows
// of the tensor-core tile and the queries in its N columns,
//
//   S^T [128 keys x N]     = Khat [128 x d] . Q^T  + A [128 x 16] . U^T
//   O^T [128 channels x N] += Vhat^T [d x 128 keys] . P^T,
//
// so that a few rows cost a few columns (N = 16..64 per group of softmax
// warps) and the softmax's work spreads over 128 threads, one per key,
// whatever the number of rows. A key behind the sequence's end is then one
// thread whose probabilities are zero.
//
// Softmax without a maximum per tile: p = 2^(s log2e - m_r + 7) is taken
// against a running maximum m_r that may trail the true one by 2^7, so p stays
// below 2^14 and keeps 21 binary orders of normal fp16 below the maximum. Only
// when a score passes m_r by more than 7 (always on a unit's first tile) the
// group takes the tile's maxima per column and rescales its sums and O. Sums
// are fp32: l in registers of the key's thread, O in TMEM.
//
// Operands are fp16 as in the chunk kernel: Khat = fp16(code s + fp16(z + mu)),
// Vhat = fp16(code s + z) with exact codes, one rounding per fp16 operation;
// queries scaled per row by a power of two, which leaves bf16 values exact;
// U = fp16 of the fp32 product of the scaled fp16 query with P in two fp16
// halves; P^T = fp16(p).
//
// Warp roles of a CTA (one per SM): 4 softmax warps per row group; 8 or 16
// producer warps (packed fields -> swizzled fp16 operand tiles, two stages;
// query tiles at the start of a unit); one warp that issues the MMAs. S^T is
// double-buffered in TMEM, so the keys of tile t + 1 are multiplied while tile
// t is in the softmax.
//
// Work: the key tiles of all units form one list (source, sequence, KV head,
// row block, tile), of which every CTA takes an equal contiguous part, found
// from the lengths on the device (a captured call replays with other lengths).
// A unit that a part's border cuts is written in pieces (unnormalised rows,
// maximum, sum) and merged by a second kernel.
//
// Every wait is bounded by an SM-clock budget; on expiry the CTA's abort flag
// ends the other waits, the workspace's first word is set, the rows of the
// CTA's remaining part become NaN and the kernel ends.
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "mbarrier.cuh"
#include "packed_tile.cuh"
#include "umma.cuh"

namespace kv2 {
namespace {

constexpr int kKeys = 128;             // keys per tile (rows of S^T)
constexpr float kBias = 7.0f;          // p = 2^(x) with x = s log2e - m + kBias
constexpr float kTrail = 14.0f;        // x above this refreshes the row's running maximum
constexpr int kStages = 2;
// A unit begins with kLead positions of the work list that hold no tile: its
// query rows, first maxima and output rows take about as long as that many key
// tiles, so parts with many short units get fewer tiles.
constexpr int kLead = 4;

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
  const uint16_t* Q;        // bf16 [rows of (b, i)][H_q][D]
  void* out;                // null: whole units go to dir_o / dir_ml
  int out_dtype;
  float scale_log2;
  int* err;
  long long* total;         // workspace: length of the work list
  long long* base;          // workspace: first position of every sequence, [src 0 | src 1]
  int4* cta;                // workspace: {source, sequence, unit in the sequence, first tile in the unit} per CTA
  float* part_o;            // pieces [CTA][2][N][D], slot 0: continues a unit, 1: begins one
  float2* part_ml;          // [CTA][2][N] running maximum and sum
  float* dir_o;             // whole units [source][rows][D]
  float2* dir_ml;
  long long dir_rows;       // rows per source of dir_*
  unsigned long long budget;
  int force_timeout;
};

// D channels, X groups of NX rows (columns of S^T), N = X * NX rows per unit
template <int D, int NX, int X>
struct RCfg {
  static constexpr int N = NX * X;
  // producer threads per key: few rows are bound by dequantization, and 16
  // warps hide its latency best; with 64 columns the softmax threads' sums
  // need the registers
  static constexpr int TPR = NX <= 32 ? 4 : 2;
  static constexpr int PW = kKeys * TPR / 32, SW = 4 * X, kMmaWarp = SW + PW;
  static constexpr int kThreads = 32 * (SW + PW + 1);
  static constexpr int CH = D / TPR;                 // channels per producer thread
  static constexpr int PB = X == 1 ? 2 : 1;          // P buffers per group
  static constexpr int Q_BYTES = NX * D * 2, U_BYTES = NX * 32, K_BYTES = kKeys * D * 2, A_BYTES = kKeys * 32;
  static constexpr int V_BYTES = kKeys * 256;        // 128 channels (zero above D)
  static constexpr int P_BYTES = NX * 256;
  static constexpr uint32_t OFF_K = 0;
  static constexpr uint32_t OFF_V = OFF_K + kStages * K_BYTES;
  static constexpr uint32_t OFF_Q = OFF_V + kStages * V_BYTES;
  static constexpr uint32_t OFF_P = OFF_Q + X * Q_BYTES;
  static constexpr uint32_t OFF_A = OFF_P + X * PB * P_BYTES;
  static constexpr uint32_t OFF_U = OFF_A + kStages * A_BYTES;
  static constexpr uint32_t OFF_FRAG = OFF_U + X * U_BYTES;             // P fragments [D/16][2][2][32] uint2
  static constexpr uint32_t OFF_SCR = OFF_FRAG + D / 16 * 2 * 2 * 32 * 8;   // row scales, ring of 4 units
  static constexpr uint32_t OFF_TAB = OFF_SCR + 4 * N * 4;              // per column pair {sc, sc, nm, nm}
  static constexpr uint32_t OFF_MROW = OFF_TAB + N * 8;
  static constexpr uint32_t OFF_ALPHA = OFF_MROW + N * 4;
  static constexpr uint32_t OFF_ROW = OFF_ALPHA + N * 4;                // row of Q and out per column
  static constexpr uint32_t OFF_RED = OFF_ROW + N * 4;                  // [X][4 warps][NX]
  static constexpr uint32_t OFF_BAR = OFF_RED + X * 4 * NX * 4;
  static constexpr uint32_t SMEM = OFF_BAR + 256 + 1024;
  static constexpr uint32_t kTmemUsed = 3 * N;
  static constexpr uint32_t kTmemCols = kTmemUsed <= 64 ? 64 : kTmemUsed <= 128 ? 128 : kTmemUsed <= 256 ? 256 : 512;
  // Q and Khat K-major; Vhat by channels; P by rows (NX = 64) or by keys
  static constexpr uint32_t kIdQK = make_idesc(0, 0, 0, NX, kKeys);
  static constexpr uint32_t kIdPV = make_idesc(0, 0, NX == 64 ? 1 : 0, NX, 128, 1);
  static_assert(SMEM <= 232448, "shared memory of one CTA");
  static_assert(NX == 16 || NX == 32 || NX == 64, "columns per group");
};
// barrier slots (bytes from OFF_BAR)
constexpr uint32_t B_KFULL = 0, B_KEMPTY = 16, B_VFULL = 32, B_VEMPTY = 48, B_SFULL = 64, B_SFREE = 96,
                   B_PFULL = 128, B_PDONE = 160, B_QFULL = 192, B_QEMPTY = 200, B_FINAL = 208, B_NEVER = 216,
                   B_TMEM = 224, B_ABORT = 228, B_PMAX = 232;

// order-preserving map of floats to signed integers, and back
__device__ __forceinline__ int f2ord(float x) {
  const int i = __float_as_int(x);
  return i ^ ((i >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float ord2f(int k) { return __int_as_float(k ^ ((k >> 31) & 0x7fffffff)); }

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
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// ---------------------------------------------------------------------------
// the work list: every unit is kLead positions, then one per key tile
// ---------------------------------------------------------------------------

// first position of CTA c of C over T positions, and the CTA that holds position u
__device__ __forceinline__ long long part_begin(long long T, int c, int C) { return T * c / C; }
__device__ __forceinline__ int part_of(long long u, long long T, int C) { return int(((u + 1) * C - 1) / T); }

struct SeqShape {
  int len, ql, nb, RB;      // keys, queries, tiles per unit, row blocks
};
template <int N>
__device__ __forceinline__ SeqShape seq_shape(const RowsSource& s, int b, int G) {
  SeqShape q;
  q.len = s.lens ? min(max(s.lens[b], 0), s.max_len) : s.max_len;
  q.ql = s.q_lens ? min(max(s.q_lens[b], 0), s.Nq) : s.Nq;
  q.nb = max(1, (q.len + kKeys - 1) / kKeys);     // an empty sequence has one masked tile: its rows become zero
  q.RB = (q.ql * G + N - 1) / N;                  // (rows fit in 30 bits)
  return q;
}

// a place in the list; every role of a CTA walks the same segments
template <int N>
struct Walk {
  long long at, hi;         // position of the unit's first tile, end of the part
  int src, b, ub, j;        // unit ub of sequence b, next tile j
  SeqShape q;
  __device__ void load(const RowsParams& p) { q = seq_shape<N>(p.src[src], b, p.H_q / p.H_kv); }
  __device__ int count() const { return int(min(static_cast<long long>(q.nb - j), hi - at - j)); }
  __device__ bool more() const { return at + j < hi; }
  __device__ int head() const { return ub / q.RB; }
  __device__ int block() const { return ub % q.RB; }
  __device__ void next(const RowsParams& p) {
    at += q.nb + kLead;
    j = 0;
    if (at >= hi) return;
    if (++ub < p.H_kv * q.RB) return;
    ub = 0;
    do {
      if (++b == p.src[src].B) {
        b = 0;
        ++src;
      }
      load(p);
    } while (q.RB == 0);
  }
};

// The list's length and this CTA's place in it, by one warp: the positions of
// 32 sequences at a time, summed by shuffles.
template <int N>
__device__ void plan(const RowsParams& p, int lane, Walk<N>& w) {
  const int G = p.H_q / p.H_kv, C = gridDim.x, c = blockIdx.x;
  long long T = 0, lo = 0;
  for (int pass = 0; pass < 2; ++pass) {
    long long at = 0;
    bool found = false;
    for (int s = 0; s < p.nsrc && !found; ++s) {
      for (int b0 = 0; b0 < p.src[s].B && !found; b0 += 32) {
        const int b = b0 + lane;
        long long v = 0;
        if (b < p.src[s].B) {
          const SeqShape q = seq_shape<N>(p.src[s], b, G);
          v = static_cast<long long>(q.nb + kLead) * q.RB * p.H_kv;
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
            const int unit = w.q.nb + kLead, in = int(rem % unit);
            w.ub = int(rem / unit);
            w.j = max(0, in - kLead);
            w.at = lo - in + kLead;
            found = true;
          }
        }
        at += __shfl_sync(0xffffffffu, inc, 31);
      }
    }
    if (pass == 0) {
      T = at;
      lo = part_begin(T, c, C);
      w.at = lo;
      w.hi = part_begin(T, c + 1, C);
      if (c == 0 && lane == 0) *p.total = T;
      if (lo >= w.hi) return;
    }
  }
}

// ---------------------------------------------------------------------------
// producers
// ---------------------------------------------------------------------------

// packed fields of CH channels of a cached token, channels part * CH ..
template <int CH>
struct Raw {
  static constexpr int W = CH / 16, Z = CH >= 64 ? 2 : 1;
  uint32_t kw[W], vw[W], ksz[Z], vsz[Z];
  int idx;
};

template <int W>
__device__ __forceinline__ void load_words(const uint32_t* src, uint32_t (&w)[W]) {
  if constexpr (W == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(src);
    w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
  } else if constexpr (W == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(src);
    w[0] = v.x; w[1] = v.y;
  } else {
    w[0] = *src;
  }
}

template <int D, int CH>
__device__ __forceinline__ void load_raw(const RowsSource& s, size_t slot, int part, Raw<CH>& r) {
  load_words<CH / 16>(s.k_code + slot * (D / 16) + part * (CH / 16), r.kw);
  load_words<CH / 16>(s.v_code + slot * (D / 16) + part * (CH / 16), r.vw);
  const size_t z = slot * (D >> s.gshift);
#pragma unroll
  for (int i = 0; i < Raw<CH>::Z; ++i) {
    const int g = (part * CH + 32 * i) >> s.gshift;
    r.ksz[i] = s.k_sz[z + g];
    r.vsz[i] = s.v_sz[z + g];
  }
  r.idx = (s.M <= 256) ? int(static_cast<const uint8_t*>(s.cidx)[slot]) : int(static_cast<const uint16_t*>(s.cidx)[slot]);
}

// the PSAC row of a cached token (fp16, zero-padded to 16 coefficients)
__device__ __forceinline__ void load_psac(const RowsSource& s, size_t slot, uint4& a0, uint4& a1) {
  a0 = a1 = make_uint4(0, 0, 0, 0);
  if (s.r == 0) return;
  if (s.psac_fmt == 1) {
    // int8 codes and the token's scale: fp16(code * scale)
    const float sc = __half2float(__ushort_as_half(s.psac_scale[slot]));
    const int8_t* q8 = reinterpret_cast<const int8_t*>(s.psac) + slot * s.r;
    const uint2 lo = *reinterpret_cast<const uint2*>(q8);
    const uint2 hi = s.r >= 16 ? *reinterpret_cast<const uint2*>(q8 + 8) : make_uint2(0, 0);
    const uint32_t w[4] = {lo.x, lo.y, hi.x, hi.y};
    uint32_t h[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t two = (w[i >> 1] >> (16 * (i & 1))) & 0xffffu;
      h[i] = pack_f16(float(int8_t(two & 0xff)) * sc, float(int8_t(two >> 8)) * sc);
    }
    a0 = make_uint4(h[0], h[1], h[2], h[3]);
    a1 = make_uint4(h[4], h[5], h[6], h[7]);
    return;
  }
  a0 = *reinterpret_cast<const uint4*>(s.psac + slot * s.r);
  if (s.r >= 16) a1 = *reinterpret_cast<const uint4*>(s.psac + slot * s.r + 8);
}

__device__ __forceinline__ uint4 dequant8(uint32_t word, int lc, uint32_t s2, const uint32_t (&add)[4]) {
  const uint32_t x = field_both(word, lc), x8 = x >> 8;
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = hfma2(code_pair_f16(x, x8, i), s2, add[i]);
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// ---------------------------------------------------------------------------
// column sums over the warp's lanes (keys): afterwards lane c % 32 holds
// column c's sum in v[c / 32] (N = 16: lanes c and c + 16)
// ---------------------------------------------------------------------------
template <int NX>
__device__ __forceinline__ void warp_colsum(float (&v)[NX], int lane) {
  constexpr int S = NX < 32 ? NX : 32;
  if constexpr (NX == 16) {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], 16);
  }
#pragma unroll
  for (int h = 0; h < NX; h += S) {
#pragma unroll
    for (int o = S / 2; o > 0; o >>= 1) {
#pragma unroll
      for (int i = 0; i < o; ++i) {
        const float a = v[h + i], b = v[h + i + o];
        const bool up = (lane & o) != 0;
        v[h + i] = (up ? b : a) + __shfl_xor_sync(0xffffffffu, up ? a : b, o);
      }
    }
    v[h / S] = v[h];
  }
}

template <int CW>
__device__ __forceinline__ void tmem_cols(uint32_t t, float (&v)[CW]) {
  if constexpr (CW == 16) {
    tmem_ld16(t, v);
  } else {
    uint32_t r[32];
    tmem_ld32_issue(t, r);
    tmem_wait_ld(r);
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
  }
}

// ---------------------------------------------------------------------------
template <int D, int NX, int X>
__global__ void __launch_bounds__(RCfg<D, NX, X>::kThreads, 1) rows_attn_kernel(const __grid_constant__ RowsParams p) {
  using Cfg = RCfg<D, NX, X>;
  constexpr int N = Cfg::N, SW = Cfg::SW, PW = Cfg::PW, PB = Cfg::PB, CH = Cfg::CH;
  constexpr int CW = NX < 32 ? NX : 32;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  const uint32_t bar = sb + Cfg::OFF_BAR;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Cfg::OFF_BAR + B_TMEM);
  volatile int* abort = reinterpret_cast<volatile int*>(smem + Cfg::OFF_BAR + B_ABORT);
  __shared__ Walk<N> walk_s;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = p.H_q / p.H_kv;

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar + B_KFULL + 8 * i, PW * 32);
      mbar_init(bar + B_KEMPTY + 8 * i, 1);
      mbar_init(bar + B_VFULL + 8 * i, PW * 32);
      mbar_init(bar + B_VEMPTY + 8 * i, 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(bar + B_SFULL + 8 * i, 1);          // [group][buffer]
      mbar_init(bar + B_SFREE + 8 * i, 128);
      mbar_init(bar + B_PFULL + 8 * i, 128);
      mbar_init(bar + B_PDONE + 8 * i, 1);
    }
    mbar_init(bar + B_QFULL, PW * 32);
    mbar_init(bar + B_QEMPTY, 1);
    mbar_init(bar + B_FINAL, 1);
    mbar_init(bar + B_NEVER, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    *abort = 0;
  }
  if (warp == Cfg::kMmaWarp) tmem_alloc(smem_u32(tmem_slot), Cfg::kTmemCols);
  if (warp == 0) {
    Walk<N> w;
    w.at = w.hi = 0;
    w.src = w.b = w.ub = w.j = 0;
    plan<N>(p, lane, w);
    if (lane == 0) {
      walk_s = w;
      p.cta[blockIdx.x] = make_int4(w.src, w.b, w.ub, w.j);
    }
  }
  if constexpr (D < 128) {
    // the channels above D of both value stages stay zero
    for (int i = tid; i < kStages * kKeys * 8; i += Cfg::kThreads)
      *reinterpret_cast<uint4*>(smem + Cfg::OFF_V + (i / (kKeys * 8)) * Cfg::V_BYTES + 16384 + (i % (kKeys * 8)) * 16) =
          make_uint4(0, 0, 0, 0);
    fence_proxy_async();
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  Walk<N> w = walk_s;

  if (warp == Cfg::kMmaWarp) {
    // ================= MMA issue (one thread) =================
    constexpr uint32_t kIdQK = Cfg::kIdQK, kIdPV = Cfg::kIdPV;
    const uint64_t dK = make_sdesc(sb + Cfg::OFF_K, 16, 1024, kLayoutSW128);
    const uint64_t dA = make_sdesc(sb + Cfg::OFF_A, 128, 256, kLayoutNone);
    const uint64_t dV = make_sdesc(sb + Cfg::OFF_V, 16384, 1024, kLayoutSW128);
    const uint64_t dQ = make_sdesc(sb + Cfg::OFF_Q, 16, 1024, kLayoutSW128);
    const uint64_t dU = make_sdesc(sb + Cfg::OFF_U, 128, 256, kLayoutNone);
    const uint64_t dP = make_sdesc(sb + Cfg::OFF_P, NX == 64 ? 16384 : 16, 1024, kLayoutSW128);
    bool ok = true;
    int t = 0, seg = 0;
    // P . V of tile t (the first of its unit's part starts the sums afresh)
    auto issue_pv = [&](int tt, bool first) -> bool {
      const int s = tt & 1;
      if (!mbar_wait_or_abort(bar + B_VFULL + 8 * s, (tt >> 1) & 1, p.budget, abort)) return false;
      for (int x = 0; x < X; ++x) {
        const int pb = PB == 2 ? (tt & 1) : 0;
        const uint32_t par = PB == 2 ? (tt >> 1) & 1 : tt & 1;
        if (!mbar_wait_or_abort(bar + B_PFULL + 16 * x + 8 * pb, par, p.budget, abort)) return false;
        fence_after_sync();
        if (lane == 0) {
          const uint32_t tO = tmem + 2 * N + x * NX;
          const uint64_t a = dV + uint64_t(s * Cfg::V_BYTES >> 4);
          const uint64_t b = dP + uint64_t((x * PB + pb) * Cfg::P_BYTES >> 4);
#pragma unroll
          for (int kk = 0; kk < kKeys / 16; ++kk) {
            const uint64_t bo = NX == 64 ? uint64_t(kk * 2048 >> 4) : uint64_t(((kk >> 2) * NX * 128 + (kk & 3) * 32) >> 4);
            mma_f16(tO, a + uint64_t(kk * 2048 >> 4), b + bo, kIdPV, !(first && kk == 0));
          }
          mma_commit(bar + B_PDONE + 16 * x + 8 * pb);
          if (x == X - 1) mma_commit(bar + B_VEMPTY + 8 * s);
        }
        __syncwarp();
      }
      return true;
    };
    bool pend = false, pend_first = false;      // tile t - 1 still waits for its P . V
    for (; ok && w.more(); ++seg) {
      const int cnt = w.count();
      const bool psac = p.src[w.src].r > 0;
      for (int jj = 0; jj < cnt; ++jj, ++t) {
        const int s = t & 1;
        ok = false;
        if (p.force_timeout && t == 0 && !mbar_wait_or_abort(bar + B_NEVER, 0, p.budget, abort)) break;
        // a unit's last P . V goes before the next unit's first tile, so that
        // its rows can be written while the next queries are multiplied
        if (jj == 0 && pend && !issue_pv(t - 1, pend_first)) break;
        if (jj == 0 && !mbar_wait_or_abort(bar + B_QFULL, seg & 1, p.budget, abort)) break;
        if (!mbar_wait_or_abort(bar + B_KFULL + 8 * s, (t >> 1) & 1, p.budget, abort)) break;
        int x = 0;
        for (; x < X; ++x) {
          if (t >= 2 && !mbar_wait_or_abort(bar + B_SFREE + 16 * x + 8 * s, ((t >> 1) - 1) & 1, p.budget, abort)) break;
          fence_after_sync();
          if (lane == 0) {
            const uint32_t tS = tmem + (x * 2 + s) * NX;
            const uint64_t a = dK + uint64_t(s * Cfg::K_BYTES >> 4), b = dQ + uint64_t(x * Cfg::Q_BYTES >> 4);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              mma_f16(tS, a + uint64_t(((kk >> 2) * 16384 + (kk & 3) * 32) >> 4),
                      b + uint64_t(((kk >> 2) * NX * 128 + (kk & 3) * 32) >> 4), kIdQK, kk > 0);
            if (psac) mma_f16(tS, dA + uint64_t(s * Cfg::A_BYTES >> 4), dU + uint64_t(x * Cfg::U_BYTES >> 4), kIdQK, 1);
            mma_commit(bar + B_SFULL + 16 * x + 8 * s);
          }
          __syncwarp();
        }
        if (x < X) break;
        if (lane == 0) {
          mma_commit(bar + B_KEMPTY + 8 * s);
          if (jj == cnt - 1) mma_commit(bar + B_QEMPTY);
        }
        __syncwarp();
        if (jj > 0 && !issue_pv(t - 1, pend_first)) break;
        pend = true;
        pend_first = jj == 0;
        ok = true;
      }
      w.next(p);
    }
    if (ok && pend) issue_pv(t - 1, pend_first);
  } else if (warp >= SW) {
    // ================= producers =================
    // lanes 8q..8q+7 of a warp take 8 consecutive keys and one part of their
    // channels: their 16-byte stores fall on 8 distinct swizzled bank groups
    const int pt = tid - SW * 32, pw = pt >> 5;
    const int row = Cfg::TPR == 4 ? pw * 8 + (lane & 7) : pw * 16 + (lane & 7) + 8 * (lane >> 4);
    const int part = Cfg::TPR == 4 ? lane >> 3 : (lane >> 3) & 1;
    uint2* frag = reinterpret_cast<uint2*>(smem + Cfg::OFF_FRAG);
    uint32_t* pmax_s = reinterpret_cast<uint32_t*>(smem + Cfg::OFF_BAR + B_PMAX);
    int t = 0, seg = 0, frag_src = -1, frag_h = -1;
    float pmax = 0.0f;
    for (; w.more(); ++seg) {
      const RowsSource& s = p.src[w.src];
      const int cnt = w.count(), h = w.head(), j0 = w.j, len = w.q.len;
      // ---- fragments of P (fp16 halves of P 2^e, max |P| 2^e in [2^13, 2^14)) for U = Q P
      if (s.r > 0 && (w.src != frag_src || h != frag_h)) {
        const float* Ph = s.P + size_t(h) * D * s.r;
        constexpr int TASKS = D / 16 * 2 * 32, PER = (TASKS + PW * 32 - 1) / (PW * 32);
        float v[PER][4];
        float mx = 0.0f;
#pragma unroll
        for (int k = 0; k < PER; ++k) {
          const int i = pt + k * PW * 32, l = i & 31, nt = (i >> 5) & 1, ks = i >> 6;
          const int n = nt * 8 + (l >> 2), c = ks * 16 + 2 * (l & 3);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            v[k][e] = (i < TASKS && n < s.r) ? Ph[size_t(c + (e & 1) + 8 * (e >> 1)) * s.r + n] : 0.0f;
            mx = fmaxf(mx, fabsf(v[k][e]));
          }
        }
        bar_sync(1, PW * 32);                     // the previous fragments and maximum are read
        if (pt == 0) *pmax_s = 0;
        bar_sync(1, PW * 32);
        const uint32_t wm = __reduce_max_sync(0xffffffffu, __float_as_uint(mx));
        if (lane == 0) atomicMax(pmax_s, wm);
        bar_sync(1, PW * 32);
        pmax = __uint_as_float(*pmax_s);
        int e2 = 0;
        if (pmax > 0.0f && pmax < 1e30f) frexpf(pmax, &e2);
        const float mul = ldexpf(1.0f, 14 - e2);
#pragma unroll
        for (int k = 0; k < PER; ++k) {
          const int i = pt + k * PW * 32, l = i & 31, nt = (i >> 5) & 1, ks = i >> 6;
          if (i >= TASKS) break;
          float hi[4], lo[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float y = v[k][e] * mul;
            hi[e] = __half2float(__float2half_rn(y));
            lo[e] = y - hi[e];
          }
          frag[((ks * 2 + nt) * 2 + 0) * 32 + l] = make_uint2(pack_f16(hi[0], hi[1]), pack_f16(hi[2], hi[3]));
          frag[((ks * 2 + nt) * 2 + 1) * 32 + l] = make_uint2(pack_f16(lo[0], lo[1]), pack_f16(lo[2], lo[3]));
        }
        bar_sync(1, PW * 32);
        frag_src = w.src;
        frag_h = h;
      }
      // ---- query rows of the unit: warp g takes rows 16 g .. 16 g + 15
      // scale 2^e per row: |q| 2^e < 2^15 and |u| = |q P| <= D max|q| max|P| likewise
      if (pw < N / 16) {
        constexpr int LPR = D / 8, RPI = 32 / LPR, IT = 16 / RPI;     // lanes per row, rows per step, steps
        const int c = lane % LPR;
        uint4 v[IT];
#pragma unroll
        for (int k = 0; k < IT; ++k) {
          const int rr = pw * 16 + k * RPI + lane / LPR;
          const int ri = w.block() * N + rr;
          v[k] = make_uint4(0, 0, 0, 0);
          if (ri < w.q.ql * G) {
            const size_t gr = (size_t(w.b) * s.Nq + ri / G) * p.H_q + h * G + ri % G;
            v[k] = __ldg(reinterpret_cast<const uint4*>(p.Q + gr * D) + c);
          }
        }
        if (seg > 0) mbar_wait_or_abort(bar + B_QEMPTY, (seg - 1) & 1, p.budget, abort);
        float* scr = reinterpret_cast<float*>(smem + Cfg::OFF_SCR) + (seg & 3) * N;
        int room = 0;                             // max(1, D max|P|) <= 2^room
        if (s.r > 0 && pmax > 0.0f && pmax < 1e30f) frexpf(fmaxf(1.0f, pmax * float(D)), &room);
#pragma unroll
        for (int k = 0; k < IT; ++k) {
          const int rr = pw * 16 + k * RPI + lane / LPR;
          const uint32_t u[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
          uint32_t am = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i) am = __vmaxu2(am, u[i] & 0x7fff7fffu);
          am = max(am & 0xffffu, am >> 16);
#pragma unroll
          for (int o = LPR / 2; o > 0; o >>= 1) am = max(am, __shfl_xor_sync(0xffffffffu, am, o));
          int qexp = 0;
          if (am > 0 && am < 0x7f80u) {           // a finite row
            int e = 0;
            frexpf(__uint_as_float(am << 16), &e);
            qexp = min(max(15 - e - room, -126), 64);
          }
          const float qmul = ldexpf(1.0f, qexp);
          uint32_t o4[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            o4[i] = pack_f16(__uint_as_float(u[i] << 16) * qmul, __uint_as_float(u[i] & 0xffff0000u) * qmul);
          const int x = rr / NX, rx = rr % NX;
          *reinterpret_cast<uint4*>(smem + Cfg::OFF_Q + x * Cfg::Q_BYTES + (c >> 3) * NX * 128 + rx * 128 +
                                    (((c & 7) ^ (rx & 7)) << 4)) = make_uint4(o4[0], o4[1], o4[2], o4[3]);
          if (c == 0) scr[rr] = p.scale_log2 * ldexpf(1.0f, -qexp);
        }
        __syncwarp();
        if (s.r > 0) {
          // U = Q P of the warp's 16 rows: fp16 query, fp16 halves of P, fp32 sums
          const int x = pw * 16 / NX, r0 = pw * 16 % NX;
          const uint32_t qb = sb + Cfg::OFF_Q + x * Cfg::Q_BYTES;
          float acc[2][4] = {};
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const int rx = r0 + (lane & 15), ck = 2 * ks + (lane >> 4);
            uint32_t a[4];
            ldsm_x4(a, qb + (ck >> 3) * NX * 128 + rx * 128 + (((ck & 7) ^ (rx & 7)) << 4));
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
              for (int hl = 0; hl < 2; ++hl) {
                const uint2 bb = frag[((ks * 2 + nt) * 2 + hl) * 32 + lane];
                mma16816(acc[nt], a, bb.x, bb.y);
              }
          }
          int e2 = 0;
          if (pmax > 0.0f && pmax < 1e30f) frexpf(pmax, &e2);
          const float back = ldexpf(1.0f, e2 - 14);
          uint8_t* ut = smem + Cfg::OFF_U + x * Cfg::U_BYTES;
#pragma unroll
          for (int nt = 0; nt < 2; ++nt) {
            const int ra = r0 + (lane >> 2), q = (lane & 3) * 4;
            *reinterpret_cast<uint32_t*>(ut + nosw_off(ra, nt) + q) = pack_f16(acc[nt][0] * back, acc[nt][1] * back);
            *reinterpret_cast<uint32_t*>(ut + nosw_off(ra + 8, nt) + q) = pack_f16(acc[nt][2] * back, acc[nt][3] * back);
          }
        }
      }
      fence_proxy_async();
      mbar_arrive(bar + B_QFULL);

      // ---- key and value tiles; the packed fields are loaded one tile ahead
      const uint4* cent4 = reinterpret_cast<const uint4*>(s.cent) + size_t(h) * s.M * (D / 8) + part * (CH / 8);
      auto slot_of = [&](int tok) { return cache_slot(s.table, s.page, p.H_kv, s.cap, w.b, h, tok); };
      Raw<CH> raw;
      bool have = j0 * kKeys + row < len;
      if (have) load_raw<D, CH>(s, slot_of(j0 * kKeys + row), part, raw);
      for (int jj = 0; jj < cnt; ++jj, ++t) {
        const int st = t & 1;
        uint4 mu[CH / 8], a0, a1;
        if (have) {
          const uint4* m4 = cent4 + size_t(min(raw.idx, s.M - 1)) * (D / 8);
#pragma unroll
          for (int c = 0; c < CH / 8; ++c) mu[c] = __ldg(m4 + c);
          if (part == 0) load_psac(s, slot_of((j0 + jj) * kKeys + row), a0, a1);
        }
        Raw<CH> next;
        const int tn = (j0 + jj + 1) * kKeys + row;
        const bool have_n = jj + 1 < cnt && tn < len;
        if (have_n) load_raw<D, CH>(s, slot_of(tn), part, next);
        uint8_t* kt = smem + Cfg::OFF_K + st * Cfg::K_BYTES;
        uint8_t* vt = smem + Cfg::OFF_V + st * Cfg::V_BYTES;
        uint8_t* at = smem + Cfg::OFF_A + st * Cfg::A_BYTES;
        if (t >= 2) mbar_wait_or_abort(bar + B_KEMPTY + 8 * st, ((t >> 1) - 1) & 1, p.budget, abort);
        if (have) {
#pragma unroll
          for (int lc = 0; lc < CH / 8; ++lc) {
            const uint32_t sz = raw.ksz[lc / 4];
            const uint32_t s2 = __byte_perm(sz, 0u, 0x1010u), z2 = __byte_perm(sz, 0u, 0x3232u);
            const uint32_t add[4] = {hadd2(z2, mu[lc].x), hadd2(z2, mu[lc].y), hadd2(z2, mu[lc].z), hadd2(z2, mu[lc].w)};
            *reinterpret_cast<uint4*>(kt + sw128_off(row, part * (CH / 8) + lc)) = dequant8(raw.kw[lc >> 1], lc, s2, add);
          }
        } else {
#pragma unroll
          for (int lc = 0; lc < CH / 8; ++lc)
            *reinterpret_cast<uint4*>(kt + sw128_off(row, part * (CH / 8) + lc)) = make_uint4(0, 0, 0, 0);
          a0 = a1 = make_uint4(0, 0, 0, 0);
        }
        if (part == 0) {
          *reinterpret_cast<uint4*>(at + nosw_off(row, 0)) = a0;
          *reinterpret_cast<uint4*>(at + nosw_off(row, 1)) = a1;
        }
        fence_proxy_async();
        mbar_arrive(bar + B_KFULL + 8 * st);
        if (t >= 2) mbar_wait_or_abort(bar + B_VEMPTY + 8 * st, ((t >> 1) - 1) & 1, p.budget, abort);
#pragma unroll
        for (int lc = 0; lc < CH / 8; ++lc) {
          uint4 o = make_uint4(0, 0, 0, 0);
          if (have) {
            const uint32_t sz = raw.vsz[lc / 4];
            const uint32_t s2 = __byte_perm(sz, 0u, 0x1010u), z2 = __byte_perm(sz, 0u, 0x3232u);
            const uint32_t add[4] = {z2, z2, z2, z2};
            o = dequant8(raw.vw[lc >> 1], lc, s2, add);
          }
          *reinterpret_cast<uint4*>(vt + sw128_off(row, part * (CH / 8) + lc)) = o;
        }
        fence_proxy_async();
        mbar_arrive(bar + B_VFULL + 8 * st);
        raw = next;
        have = have_n;
      }
      w.next(p);
    }
  } else {
    // ================= softmax of row group x (thread = key = TMEM lane) =================
    const int x = warp >> 2, wq = warp & 3, kl = wq * 32 + lane, bid = 2 + x;
    const uint32_t lane_base = uint32_t(wq * 32) << 16;
    const uint32_t tO = tmem + 2 * N + x * NX + lane_base;
    float4* tab = reinterpret_cast<float4*>(smem + Cfg::OFF_TAB) + x * (NX / 2);
    float* tabf = reinterpret_cast<float*>(tab);
    float* mrow = reinterpret_cast<float*>(smem + Cfg::OFF_MROW) + x * NX;
    float* alpha = reinterpret_cast<float*>(smem + Cfg::OFF_ALPHA) + x * NX;
    int* row_s = reinterpret_cast<int*>(smem + Cfg::OFF_ROW) + x * NX;
    float* red = reinterpret_cast<float*>(smem + Cfg::OFF_RED) + x * 4 * NX;
    auto wait_pv = [&](int tt) {                // P . V of tile tt is complete
      const int pb = PB == 2 ? (tt & 1) : 0;
      return mbar_wait_or_abort(bar + B_PDONE + 16 * x + 8 * pb, PB == 2 ? (tt >> 1) & 1 : tt & 1, p.budget, abort);
    };
    float l[NX];
#pragma unroll
    for (int c = 0; c < NX; ++c) l[c] = 0.0f;
    bool dead = false;                          // a wait ran out (seen by this thread)
    bool gone = false;                          // ... by the group
    int t = 0, seg = 0;
    for (; w.more(); ++seg) {
      const RowsSource& s = p.src[w.src];
      const int cnt = w.count(), j0 = w.j, len = w.q.len, h = w.head();
      const float* scr = reinterpret_cast<const float*>(smem + Cfg::OFF_SCR) + (seg & 3) * N + x * NX;
      for (int jj = 0; jj < cnt && !gone; ++jj, ++t) {
        const int sbuf = t & 1;
        const uint32_t tS = tmem + (x * 2 + sbuf) * NX + lane_base;
        dead |= !mbar_wait_or_abort(bar + B_SFULL + 16 * x + 8 * sbuf, (t >> 1) & 1, p.budget, abort);
        fence_after_sync();
        const int k0 = (j0 + jj) * kKeys;
        const bool valid = k0 + kl < len;
        bool refresh = true;
        if (jj == 0) {
          if (kl < NX) {
            mrow[kl] = -INFINITY;
          }
#pragma unroll
          for (int c = 0; c < NX; ++c) l[c] = 0.0f;
        } else {
          // does a score pass its row's running maximum by more than the margin?
          float mx = -INFINITY;
#pragma unroll
          for (int c0 = 0; c0 < NX; c0 += CW) {
            float v[CW];
            tmem_cols<CW>(tS + c0, v);
#pragma unroll
            for (int i = 0; i < CW; i += 2) {
              const float4 k = tab[(c0 + i) >> 1];
              const float2 xx = up2(ffma2(pk2(v[i], v[i + 1]), pk2(k.x, k.y), pk2(k.z, k.w)));
              mx = fmax3(mx, xx.x, xx.y);
            }
          }
          refresh = bar_or(bid, 128, (valid && mx > kTrail) || dead);
        }
        if (refresh) {
          if (bar_or(bid, 128, dead)) { gone = true; break; }
#pragma unroll
          for (int c0 = 0; c0 < NX; c0 += CW) {
            float v[CW];
            tmem_cols<CW>(tS + c0, v);
            int mine = 0;
#pragma unroll
            for (int i = 0; i < CW; ++i) {
              const float sv = valid ? v[i] * scr[c0 + i] : -INFINITY;
              const int m = __reduce_max_sync(0xffffffffu, f2ord(sv));
              if (lane == i) mine = m;
            }
            if (lane < CW) red[wq * NX + c0 + lane] = ord2f(mine);
          }
          // O is rescaled below: P . V of the tile before must be complete
          if (jj > 0) dead |= !wait_pv(t - 1);
          fence_after_sync();
          bar_sync(bid, 128);
          if (kl < NX) {
            const float tm = fmaxf(fmaxf(red[kl], red[NX + kl]), fmaxf(red[2 * NX + kl], red[3 * NX + kl]));
            // A whole number: every rescaling is by an exact power of two, and
            // p's rounding does not depend on where the work is cut. Only the
            // rows that need it: a row's result does not depend on the others.
            const float mo = mrow[kl], mn = tm > mo + (kTrail - kBias) ? ceilf(tm) : mo;
            alpha[kl] = mn == -INFINITY ? 1.0f : ex2(mo - mn);
            mrow[kl] = mn;
            // s sc - m is one fma, exact to half a step of m: beyond 2^20 (where
            // a key's fp16 rounding already moves the score by 2^8) the row's
            // scores are taken at a 2^-k of their size, so that this stays small
            int e = 0;
            if (fabsf(mn) > 0x1p20f && fabsf(mn) < INFINITY) frexpf(mn, &e);
            const float damp = ldexpf(1.0f, -max(e - 21, 0));
            tabf[(kl >> 1) * 4 + (kl & 1)] = scr[kl] * damp;
            tabf[(kl >> 1) * 4 + 2 + (kl & 1)] = mn == -INFINITY ? 0.0f : kBias - mn * damp;
          }
          bar_sync(bid, 128);
          if (jj > 0) {
#pragma unroll
            for (int c = 0; c < NX; ++c) l[c] *= alpha[c];
#pragma unroll
            for (int c0 = 0; c0 < NX; c0 += 16) {
              float v[16];
              uint32_t o[16];
              tmem_ld16(tO + c0, v);
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(v[i] * alpha[c0 + i]);
              tmem_st16(tO + c0, o);
            }
            tmem_wait_st();
          }
        }
        // ---- probabilities into the P operand, once its buffer is free
        if (t >= PB) dead |= !wait_pv(t - PB);
        uint8_t* pt8 = smem + Cfg::OFF_P + (x * PB + (PB == 2 ? sbuf : 0)) * Cfg::P_BYTES;
        const bool full = k0 + kKeys <= len;
#pragma unroll
        for (int c0 = 0; c0 < NX; c0 += CW) {
          float v[CW];
          tmem_cols<CW>(tS + c0, v);
          if (c0 + CW == NX) {                    // the scores are in registers: the buffer may be rewritten
            fence_before_sync();
            mbar_arrive(bar + B_SFREE + 16 * x + 8 * sbuf);
          }
          uint32_t pw2[CW / 2];
#pragma unroll
          for (int i = 0; i < CW; i += 2) {
            const float4 k = tab[(c0 + i) >> 1];
            const float2 xx = up2(ffma2(pk2(v[i], v[i + 1]), pk2(k.x, k.y), pk2(k.z, k.w)));
            float p0 = ex2(xx.x), p1 = ex2(xx.y);
            if (!full) {
              p0 = valid ? p0 : 0.0f;
              p1 = valid ? p1 : 0.0f;
            }
            l[c0 + i] += p0;
            l[c0 + i + 1] += p1;
            pw2[i / 2] = pack_f16(p0, p1);
          }
          if constexpr (NX == 64) {
            // rows along the operand's contiguous dimension: [key][64 rows], swizzled
#pragma unroll
            for (int i = 0; i < CW / 8; ++i)
              *reinterpret_cast<uint4*>(pt8 + kl * 128 + (((c0 / 8 + i) ^ (kl & 7)) << 4)) =
                  make_uint4(pw2[4 * i], pw2[4 * i + 1], pw2[4 * i + 2], pw2[4 * i + 3]);
          } else {
            // keys along the contiguous dimension: [2][row][64 keys], swizzled
#pragma unroll
            for (int i = 0; i < CW; ++i) {
              const int rr = c0 + i;
              *reinterpret_cast<uint16_t*>(pt8 + (kl >> 6) * NX * 128 + rr * 128 + ((((kl & 63) >> 3) ^ (rr & 7)) << 4) +
                                           (kl & 7) * 2) = uint16_t((i & 1) ? pw2[i / 2] >> 16 : pw2[i / 2] & 0xffffu);
            }
          }
        }
        fence_proxy_async();
        fence_before_sync();
        mbar_arrive(bar + B_PFULL + 16 * x + 8 * (PB == 2 ? sbuf : 0));
      }
      // ---- the unit's rows
      if (!gone) {
        dead |= !wait_pv(t - 1);
        fence_after_sync();
        gone = bar_or(bid, 128, dead);
      }
      warp_colsum<NX>(l, lane);
      if (NX >= 32 || lane < NX) {
#pragma unroll
        for (int c = 0; c < (NX + 31) / 32; ++c) red[wq * NX + c * 32 + lane] = l[c];
      }
      bar_sync(bid, 128);
      const bool whole = j0 == 0 && cnt == w.q.nb;
      const int slot = j0 > 0 ? 0 : 1;
      const int r0 = w.block() * N + x * NX, live = min(NX, w.q.ql * G - r0);
      if (kl < NX) {
        float lt = (red[kl] + red[NX + kl]) + (red[2 * NX + kl] + red[3 * NX + kl]);
        float m = mrow[kl];
        if (gone) {
          lt = 1.0f;
          m = 0.0f;
        }
        alpha[kl] = lt > 0.0f ? 1.0f / lt : (lt == 0.0f ? 0.0f : lt);
        if (kl < live) {
          // row of (sequence, query, head) in Q and out
          const int ri = r0 + kl, row = (w.b * s.Nq + ri / G) * p.H_q + h * G + ri % G;
          row_s[kl] = row;
          if (!whole) p.part_ml[(size_t(blockIdx.x) * 2 + slot) * N + x * NX + kl] = make_float2(m, lt);
          else if (!p.out) p.dir_ml[size_t(w.src) * p.dir_rows + row] = make_float2(m, lt);
        }
      }
      bar_sync(bid, 128);
#pragma unroll 1
      for (int c0 = 0; c0 < NX; c0 += 16) {
        if (c0 >= live) break;
        float v[16];
        if (!gone) {
          tmem_ld16(tO + c0, v);                  // every lane: warp-wide TMEM load
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = __int_as_float(0x7fc00000);
        }
        if (kl < D) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int c = c0 + i;
            if (c >= live) break;
            if (!whole) {
              p.part_o[((size_t(blockIdx.x) * 2 + slot) * N + x * NX + c) * D + kl] = v[i];
            } else if (!p.out) {
              p.dir_o[(size_t(w.src) * p.dir_rows + row_s[c]) * D + kl] = v[i];
            } else {
              const float o = v[i] * alpha[c];
              const size_t at = size_t(row_s[c]) * D + kl;
              if (p.out_dtype == KV2_OUT_F32) static_cast<float*>(p.out)[at] = o;
              else static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(o);
            }
          }
        }
      }
      w.next(p);
    }
  }

  // the merge (this grid's programmatic dependent) may be scheduled; it waits
  // for this grid before it reads anything
  asm volatile("griddepcontrol.launch_dependents;");
  fence_before_sync();
  __syncthreads();
  if (warp == Cfg::kMmaWarp) {
    if (*abort) {
      if (lane == 0) {
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

// One warp: log-sum-exp of one row's pieces, those of CTAs c0 (slot 1) and
// c0 + 1 .. c1 (slot 0); lane i holds channels i, i + 32, ...
template <int D>
__device__ __forceinline__ void merge_pieces(const float* part_o, const float2* part_ml, int N, int row, int c0, int c1,
                                            long long T, int C, int lane, float& m, float& l, float (&o)[D / 32]) {
  m = -INFINITY;
  for (int s0 = c0; s0 <= c1; s0 += 32) {
    const int c = s0 + lane;
    if (c <= c1 && part_begin(T, c, C) < part_begin(T, c + 1, C)) {
      const float2 ml = part_ml[(size_t(c) * 2 + (c == c0)) * N + row];
      if (!(ml.y == 0.0f)) m = fmaxf(m, ml.x);
    }
  }
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
  l = 0.0f;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) o[i] = 0.0f;
  for (int s0 = c0; s0 <= c1; s0 += 32) {
    const int c = s0 + lane;
    float f = 0.0f;
    if (c <= c1 && part_begin(T, c, C) < part_begin(T, c + 1, C)) {
      const float2 ml = part_ml[(size_t(c) * 2 + (c == c0)) * N + row];
      if (!(ml.y == 0.0f)) {
        f = exp2f(ml.x - m);
        l = fmaf(f, ml.y, l);
      }
    }
    const int n = min(32, c1 - s0 + 1);
#pragma unroll 4
    for (int k = 0; k < n; ++k) {
      const float fk = __shfl_sync(0xffffffffu, f, k);
      if (fk == 0.0f) continue;                   // an empty or absent piece (uniform over the warp)
      const float* po = part_o + ((size_t(s0 + k) * 2 + (s0 + k == c0)) * N + row) * D;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) o[i] = fmaf(fk, po[i * 32 + lane], o[i]);
    }
  }
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) l += __shfl_xor_sync(0xffffffffu, l, k);
}

template <int D>
__device__ __forceinline__ void store_row(void* out, int out_dtype, size_t row, int lane, float l, const float (&o)[D / 32]) {
  const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    const size_t at = row * D + i * 32 + lane;
    if (out_dtype == KV2_OUT_F32) static_cast<float*>(out)[at] = o[i] * inv;
    else static_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16_rn(o[i] * inv);
  }
}

// One source: block (c - 1, .) merges the unit that the border before CTA c
// cuts, if it is the unit's first border; one warp per row.
template <int D, int N>
__global__ void __launch_bounds__(256) rows_merge_cut(const __grid_constant__ RowsParams p, int C) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c = blockIdx.x + 1, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long T = *p.total, lo = part_begin(T, c, C);
  if (lo >= part_begin(T, c + 1, C)) return;
  const int4 at = p.cta[c];
  if (at.w == 0) return;                          // no unit is cut here
  const int G = p.H_q / p.H_kv;
  const SeqShape q = seq_shape<N>(p.src[0], at.y, G);
  const long long u = lo - at.w;                  // position of the unit's first tile
  const int c0 = part_of(u, T, C), c1 = part_of(u + q.nb - 1, T, C);
  if (part_begin(T, c0 + 1, C) != lo) return;     // an earlier border of the same unit
  const int row = blockIdx.y * 8 + warp;
  const int ri = (at.z % q.RB) * N + row;
  if (ri >= q.ql * G) return;
  float m, l, o[D / 32];
  merge_pieces<D>(p.part_o, p.part_ml, N, row, c0, c1, T, C, lane, m, l, o);
  const size_t gr = (size_t(at.y) * p.src[0].Nq + ri / G) * p.H_q + (at.z / q.RB) * G + ri % G;
  store_row<D>(p.out, p.out_dtype, gr, lane, l, o);
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
  float m[2], l[2], o[2][D / 32];
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const RowsSource& src = p.src[s];
    const int seq = int(gr / p.H_q), b = seq / src.Nq, i = seq % src.Nq;
    const SeqShape q = seq_shape<N>(src, b, G);
    const int ri = i * G + g;
    const long long u = p.base[(s ? p.src[0].B : 0) + b] +
                        (static_cast<long long>(h) * q.RB + ri / N) * (q.nb + kLead) + kLead;
    const int c0 = part_of(u, T, C), c1 = part_of(u + q.nb - 1, T, C);
    if (c0 == c1) {
      const float2 ml = p.dir_ml[size_t(s) * p.dir_rows + gr];
      m[s] = ml.x;
      l[s] = ml.y;
#pragma unroll
      for (int k = 0; k < D / 32; ++k) o[s][k] = p.dir_o[(size_t(s) * p.dir_rows + gr) * D + k * 32 + lane];
    } else {
      merge_pieces<D>(p.part_o, p.part_ml, N, ri % N, c0, c1, T, C, lane, m[s], l[s], o[s]);
    }
  }
  const float mm = fmaxf(l[0] == 0.0f ? -INFINITY : m[0], l[1] == 0.0f ? -INFINITY : m[1]);
  const float f0 = l[0] == 0.0f ? 0.0f : exp2f(m[0] - mm), f1 = l[1] == 0.0f ? 0.0f : exp2f(m[1] - mm);
  float r[D / 32];
#pragma unroll
  for (int k = 0; k < D / 32; ++k) r[k] = (f0 == 0.0f ? 0.0f : f0 * o[0][k]) + (f1 == 0.0f ? 0.0f : f1 * o[1][k]);
  store_row<D>(p.out, p.out_dtype, size_t(gr), lane, f0 * l[0] + f1 * l[1], r);
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
int unit_rows(long long rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128; }

// workspace: header (word 0 the error word, the tile count at byte 16), the
// first tile of every sequence, the CTAs' places, pieces, whole units
struct RowsPlan {
  int N, C;
  long long rows;
  size_t base, cta, part_ml, part_o, dir_ml, dir_o, bytes;
};
size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

RowsPlan plan_rows(const RowsArgs& a) {
  RowsPlan pl{};
  const int G = a.H_q / a.src[0].c->H_kv, d = a.src[0].c->d;
  long long most = 0;
  for (int s = 0; s < a.nsrc; ++s) most = std::max(most, static_cast<long long>(a.src[s].Nq) * G);
  pl.N = unit_rows(most);
  long long tiles = 0;
  size_t seqs = 0;
  for (int s = 0; s < a.nsrc; ++s) {
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
  pl.dir_o = pl.dir_ml + (a.nsrc == 2 ? up256(size_t(2) * pl.rows * 8) : 0);
  pl.bytes = pl.dir_o + (a.nsrc == 2 ? up256(size_t(2) * pl.rows * d * 4) : 0);
  return pl;
}

template <int D, int NX, int X>
cudaError_t launch_cfg(const RowsParams& p, const RowsPlan& pl, cudaStream_t s) {
  using Cfg = RCfg<D, NX, X>;
  auto kern = rows_attn_kernel<D, NX, X>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(Cfg::SMEM));
  if (e != cudaSuccess) return e;
  RowsParams q = p;
  if (p.nsrc == 2) q.out = nullptr;
  kern<<<pl.C, Cfg::kThreads, Cfg::SMEM, s>>>(q);
  e = cudaGetLastError();
  if (e != cudaSuccess || (p.nsrc == 1 && pl.C == 1)) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = p.nsrc == 2 ? dim3(unsigned((pl.rows + 7) / 8)) : dim3(pl.C - 1, Cfg::N / 8);
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, p.nsrc == 2 ? rows_merge_shared<D, Cfg::N> : rows_merge_cut<D, Cfg::N>, p, pl.C);
}

template <int D>
cudaError_t launch_d(const RowsParams& p, const RowsPlan& pl, cudaStream_t s) {
  switch (pl.N) {
    case 16: return launch_cfg<D, 16, 1>(p, pl, s);
    case 32: return launch_cfg<D, 32, 1>(p, pl, s);
    case 64: return launch_cfg<D, 64, 1>(p, pl, s);
    default: return launch_cfg<D, 64, 2>(p, pl, s);
  }
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
  p.nsrc = a.nsrc;
  p.H_kv = a.src[0].c->H_kv;
  p.H_q = a.H_q;
  p.Q = a.Q;
  p.out = a.out;
  p.out_dtype = a.out_dtype;
  p.scale_log2 = a.sm_scale * 1.4426950408889634f;
  p.err = reinterpret_cast<int*>(ws);
  p.total = reinterpret_cast<long long*>(ws + 16);
  p.base = reinterpret_cast<long long*>(ws + pl.base);
  p.cta = reinterpret_cast<int4*>(ws + pl.cta);
  p.part_ml = reinterpret_cast<float2*>(ws + pl.part_ml);
  p.part_o = reinterpret_cast<float*>(ws + pl.part_o);
  p.dir_ml = reinterpret_cast<float2*>(ws + pl.dir_ml);
  p.dir_o = reinterpret_cast<float*>(ws + pl.dir_o);
  p.dir_rows = pl.rows;
  p.force_timeout = env_force_timeout();
  p.budget = p.force_timeout ? (1ull << 20) : env_wait_budget();
  return a.src[0].c->d == 64 ? launch_d<64>(p, pl, s) : launch_d<128>(p, pl, s);
}

}  // namespace kv2
