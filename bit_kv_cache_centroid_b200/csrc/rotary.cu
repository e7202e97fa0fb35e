// rotary.cu — appending keys and values to the packed cache at per-sequence
// places, with the position rotation applied to keys and queries on the way.
//
// A channel pair (a, b) of a token at position p turns by the table's angles,
//   a' = a cos - b sin,   b' = b cos + a sin,
// in fp32 with every product and sum rounded (no fused multiply-add, so that
// the rotated key is the same wherever it is computed), then rounded once to
// bf16: the key that "QuantWM: Training-Free 2-bit KV Cache Quantization for
// Stable Video World Models", "1. QSAC" quantizes is the one attention reads.
//
// Two kernels. rotate_rows: one block per token of the padded batch turns the
// token's keys (to the workspace, tokens in use packed together) and queries,
// codes its values into the cache, and notes where the token goes; quantize_kernel
// (quantize.cuh), its programmatic dependent, then quantizes the packed keys as
// every append does. Tokens behind a sequence's count cost an empty block.
//
// Bound: memory; per token and KV head 256 B of key read, 256 B written and
// read back (L2 for appends below its size), 256 B of values read, and per
// query head 512 B (d = 128). A token's chain of reads (count, place, page,
// angles, rows) is long and its bytes few, so that many small blocks hide it
// best: D / 8 lanes take a head row, each its 8 channels of every head with
// the angles in registers, which leaves 32 registers a thread and 8 blocks an
// SM. Measured against 48 registers (5 blocks), 2 or 4 heads' loads in flight
// and several tokens a block: 75 us the append of up to 6 x 777 tokens (8 KV,
// 32 query heads) against 77 to 90, of which the key kernel takes 50.
#include "codec.cuh"
#include "common.cuh"
#include "internal.h"

namespace kv2 {
namespace {

constexpr int kThreads = 256;
constexpr size_t kWsHeader = 256;       // word 0: the sticky error word; word 4: rows in use

struct RotateParams {
  RotaryArgs a;
  int B, H, cap, page;
  const int32_t* table;
  uint32_t* v_code;
  uint32_t* v_sz;
  uint16_t* Kr;        // rotated keys of the rows in use, [row][H][D]
  int2* rows;          // their places
  int* n_rows;
  int* err;
};

__device__ __forceinline__ float bf(uint32_t bits) { return __uint_as_float(bits << 16); }   // the low half
__device__ __forceinline__ uint16_t bf_rn(float x) { return __bfloat16_as_ushort(__float2bfloat16_rn(x)); }
__device__ __forceinline__ void turn(float a, float b, float c, float s, float& x, float& y) {
  x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  y = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
}
// two turned pairs of bf16: (a, b) in, (a', b') out
__device__ __forceinline__ void turn2(uint32_t& a, uint32_t& b, float2 c, float2 n) {
  float x0, y0, x1, y1;
  turn(bf(a), bf(b), c.x, n.x, x0, y0);
  turn(__uint_as_float(a & 0xffff0000u), __uint_as_float(b & 0xffff0000u), c.y, n.y, x1, y1);
  const __nv_bfloat162 p = __floats2bfloat162_rn(x0, x1), q = __floats2bfloat162_rn(y0, y1);
  a = *reinterpret_cast<const uint32_t*>(&p);
  b = *reinterpret_cast<const uint32_t*>(&q);
}

// A lane's 8 channels of every head of a token: four pairs of the rotated
// channels, or 8 plain ones behind them (rot a multiple of 8). D / 8 lanes
// share a head row; the pairs' angles stay in registers from head to head.
struct LaneTurn {
  float4 c, n;
  int lo, hi;           // its two runs of four channels
  bool turned, inter;
  __device__ LaneTurn(const float* cs, int rot, int interleaved, int i) : inter(interleaved != 0) {
    const int half = rot >> 1;
    turned = 8 * i < rot;
    lo = turned && !inter ? 4 * i : 8 * i;
    hi = turned && !inter ? half + 4 * i : 8 * i + 4;
    if (turned) {
      c = __ldg(reinterpret_cast<const float4*>(cs + 4 * i));
      n = __ldg(reinterpret_cast<const float4*>(cs + half + 4 * i));
    }
  }
  // reads all it writes before it writes: dst may be src
  __device__ void run(const uint16_t* src, uint16_t* dst) const {
    uint2 a = *reinterpret_cast<const uint2*>(src + lo), b = *reinterpret_cast<const uint2*>(src + hi);
    if (turned) {
      if (inter) {                               // neighbours apart, and back below
        const uint2 t = a;
        a = make_uint2(__byte_perm(t.x, t.y, 0x5410), __byte_perm(b.x, b.y, 0x5410));
        b = make_uint2(__byte_perm(t.x, t.y, 0x7632), __byte_perm(b.x, b.y, 0x7632));
      }
      turn2(a.x, b.x, make_float2(c.x, c.y), make_float2(n.x, n.y));
      turn2(a.y, b.y, make_float2(c.z, c.w), make_float2(n.z, n.w));
      if (inter) {
        const uint2 t = a;
        a = make_uint2(__byte_perm(t.x, b.x, 0x5410), __byte_perm(t.x, b.x, 0x7632));
        b = make_uint2(__byte_perm(t.y, b.y, 0x5410), __byte_perm(t.y, b.y, 0x7632));
      }
    }
    *reinterpret_cast<uint2*>(dst + lo) = a;
    *reinterpret_cast<uint2*>(dst + hi) = b;
  }
};

template <int D, int GS>
__global__ void __launch_bounds__(kThreads, 8) rotate_rows(RotateParams p) {
  constexpr int NG = D / GS;
  __shared__ int before_s[kThreads / 32];
  // the key kernel may be scheduled; it waits for this grid before it reads
  asm volatile("griddepcontrol.launch_dependents;");
  const RotaryArgs& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / a.n_new, t = blockIdx.x % a.n_new;
  auto count_of = [&](int s) { return a.count ? min(max(a.count[s], 0), a.n_new) : a.n_new; };
  const int mine = count_of(b);
  const bool last = b == p.B - 1 && t == a.n_new - 1;
  if (t >= mine && !last) return;
  // rows of the sequences before this one
  int before = 0;
  if (a.count) {
    for (int s = tid; s < b; s += kThreads) before += count_of(s);
    before = __reduce_add_sync(0xffffffffu, before);
    if (lane == 0) before_s[warp] = before;
    __syncthreads();
    before = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) before += before_s[w];
  } else {
    before = b * a.n_new;
  }
  if (last && tid == 0) *p.n_rows = before + mine;
  if (t >= mine) return;

  // where the token goes: a slot of the cache, and a row of the table
  const long long slot = static_cast<long long>(a.start[b]) + t;
  const int pos = a.position[size_t(b) * a.n_new + t];
  const bool turned = pos >= 0 && pos < a.positions;
  int lead = -1, off = 0;
  if (turned && slot >= 0 && slot < p.cap) {
    lead = b;
    off = int(slot);
    if (p.table) {
      lead = p.table[size_t(b) * (p.cap / p.page) + off / p.page];
      off %= p.page;
    }
  }
  const int row = before + t;
  if (tid == 0) {
    p.rows[row] = make_int2(lead < 0 ? -1 : lead, off);
    if (lead < 0) atomicExch(p.err, 1);
  }
  const size_t tok = size_t(b) * a.n_new + t;
  if (!turned) {
    // no such angle: the token is not stored and its queries are not numbers
    if (a.Q)
      for (int i = tid; i < a.H_q * D; i += kThreads) a.Q_out[tok * a.H_q * D + i] = 0x7fc0u;
    return;
  }
  const float* cs = a.cos_sin + size_t(pos) * a.rot;
  const int nk = lead < 0 ? 0 : p.H, heads = nk + (a.Q ? a.H_q : 0);
  constexpr int NL = D / 8, ROWS = kThreads / NL;   // lanes of a head row, rows at a time
  const int part = tid % NL, h0 = tid / NL;
  auto from = [&](int h) { return h < nk ? a.K + (tok * p.H + h) * D : a.Q + (tok * a.H_q + (h - nk)) * D; };
  auto to = [&](int h) { return h < nk ? p.Kr + (size_t(row) * p.H + h) * D : a.Q_out + (tok * a.H_q + (h - nk)) * D; };
  if (a.rot % 8 == 0) {
    const LaneTurn lt(cs, a.rot, a.interleaved, part);
    for (int h = h0; h < heads; h += ROWS) lt.run(from(h), to(h));
  } else {
    // any even rot: a pair or a plain channel at a time
    const int half = a.rot >> 1;
#pragma unroll 1
    for (int h = h0; h < heads; h += ROWS) {
      const uint16_t* src = from(h);
      uint16_t* dst = to(h);
#pragma unroll 1
      for (int j = part; j < D - half; j += NL) {
        if (j >= half) {
          dst[j + half] = src[j + half];
          continue;
        }
        const int ca = a.interleaved ? 2 * j : j, cb = a.interleaved ? 2 * j + 1 : j + half;
        float x, y;
        turn(bf(src[ca]), bf(src[cb]), __ldg(cs + j), __ldg(cs + half + j), x, y);
        dst[ca] = bf_rn(x);
        dst[cb] = bf_rn(y);
      }
    }
  }
  if (lead < 0) return;
  // ---- values: 8 channels a lane (every lane takes part in the shuffles)
  for (int w0 = warp * (32 / NL); w0 < p.H; w0 += ROWS) {
    const int h = w0 + lane / NL;
    const bool live = h < p.H;
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (live) v = *(reinterpret_cast<const uint4*>(a.V + (tok * p.H + h) * D) + part);
    uint32_t bits;
    const GroupParams gp = code_values8<GS>(v, bits);
    if (live) {
      const size_t at = (size_t(lead) * p.H + h) * size_t(p.table ? p.page : p.cap) + off;
      reinterpret_cast<uint16_t*>(p.v_code)[at * NL + part] = uint16_t(bits);
      if (part % (GS / 8) == 0) p.v_sz[at * NG + part / (GS / 8)] = uint32_t(gp.s_bits) | (uint32_t(gp.z_bits) << 16);
    }
  }
}

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }
size_t rows_bytes(const kv2_cache& c, int n_new) { return up256(size_t(c.B) * n_new * sizeof(int2)); }

}  // namespace

size_t rotary_workspace_bytes(const kv2_cache& c, int n_new) {
  return kWsHeader + rows_bytes(c, n_new) + size_t(c.B) * n_new * c.H_kv * c.d * 2;
}

cudaError_t launch_rotary(const RotaryArgs& a, const QuantizeArgs& q, cudaStream_t s) {
  const kv2_cache& c = *a.c;
  char* ws = static_cast<char*>(a.ws);
  RotateParams p{};
  p.a = a;
  p.B = c.B; p.H = c.H_kv; p.cap = c.capacity; p.page = c.page_tokens;
  p.table = c.block_table;
  p.v_code = c.v_code;
  p.v_sz = c.v_sz;
  p.err = reinterpret_cast<int*>(ws);
  p.n_rows = reinterpret_cast<int*>(ws + 16);
  p.rows = reinterpret_cast<int2*>(ws + kWsHeader);
  p.Kr = reinterpret_cast<uint16_t*>(ws + kWsHeader + rows_bytes(c, a.n_new));
  const unsigned grid = unsigned(c.B) * unsigned(a.n_new);
  switch (q.group + c.d) {
    case 32 + 64: rotate_rows<64, 32><<<grid, kThreads, 0, s>>>(p); break;
    case 64 + 64: rotate_rows<64, 64><<<grid, kThreads, 0, s>>>(p); break;
    case 32 + 128: rotate_rows<128, 32><<<grid, kThreads, 0, s>>>(p); break;
    case 64 + 128: rotate_rows<128, 64><<<grid, kThreads, 0, s>>>(p); break;
    case 128 + 128: rotate_rows<128, 128><<<grid, kThreads, 0, s>>>(p); break;
    default: return cudaErrorInvalidValue;
  }
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  QuantizeArgs k = q;
  k.K = p.Kr;
  k.V = nullptr;
  k.rows = p.rows;
  k.n_rows = p.n_rows;
  return launch_quantize_rows(k, s);
}

}  // namespace kv2
