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
// (quantize.cu), its programmatic dependent, then quantizes the packed keys as
// every append does. Tokens behind a sequence's count cost an empty block.
//
// Bound: memory; per token and KV head 256 B of key read, 256 B written and
// read back (L2 for appends below its size), 256 B of values read, and per
// query head 512 B (d = 128).
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

__device__ __forceinline__ float bf(uint32_t bits) { return __uint_as_float(bits << 16); }
__device__ __forceinline__ uint16_t bf_rn(float x) { return __bfloat16_as_ushort(__float2bfloat16_rn(x)); }
__device__ __forceinline__ void turn(float a, float b, float c, float s, float& x, float& y) {
  x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  y = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  return uint32_t(bf_rn(a)) | (uint32_t(bf_rn(b)) << 16);
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 x = __ldg(reinterpret_cast<const float4*>(p)), y = __ldg(reinterpret_cast<const float4*>(p) + 1);
  v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
  v[4] = y.x; v[5] = y.y; v[6] = y.z; v[7] = y.w;
}

// One head row of D channels: task i of `tasks(rot)`. A task reads all it
// writes before writing, so dst may be src.
//   rot a multiple of 16, halves: chunks of 8 pairs, then chunks of 8 plain channels
//   rot a multiple of 16, neighbours: chunks of 8 channels
//   else: single pairs, then single plain channels
template <int D>
struct RowTurn {
  const float* cs;      // the position's row: rot/2 cosines, rot/2 sines
  int rot, inter;
  __device__ int tasks() const {
    if (rot & 15) return D - rot / 2;
    return inter ? D / 8 : D / 8 - rot / 16;
  }
  __device__ void run(const uint16_t* src, uint16_t* dst, int i) const {
    const int half = rot >> 1;
    if (rot & 15) {
      if (i >= half) {
        dst[i + half] = src[i + half];
        return;
      }
      const int ca = inter ? 2 * i : i, cb = inter ? 2 * i + 1 : i + half;
      float x, y;
      turn(bf(src[ca]), bf(src[cb]), __ldg(cs + i), __ldg(cs + half + i), x, y);
      dst[ca] = bf_rn(x);
      dst[cb] = bf_rn(y);
      return;
    }
    const uint4* s4 = reinterpret_cast<const uint4*>(src);
    uint4* d4 = reinterpret_cast<uint4*>(dst);
    if (inter) {
      const uint4 v = s4[i];
      uint32_t w[4] = {v.x, v.y, v.z, v.w};
      if (8 * i < rot) {
        const float4 c4 = __ldg(reinterpret_cast<const float4*>(cs + 4 * i));
        const float4 n4 = __ldg(reinterpret_cast<const float4*>(cs + half + 4 * i));
        const float c[4] = {c4.x, c4.y, c4.z, c4.w}, n[4] = {n4.x, n4.y, n4.z, n4.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float x, y;
          turn(bf(w[k] & 0xffffu), bf(w[k] >> 16), c[k], n[k], x, y);
          w[k] = pack2(x, y);
        }
      }
      d4[i] = make_uint4(w[0], w[1], w[2], w[3]);
      return;
    }
    if (i >= rot / 16) {
      d4[i + rot / 16] = s4[i + rot / 16];
      return;
    }
    const uint4 va = s4[i], vb = s4[i + rot / 16];
    const uint32_t a[4] = {va.x, va.y, va.z, va.w}, b[4] = {vb.x, vb.y, vb.z, vb.w};
    float c[8], n[8];
    load8(cs + 8 * i, c);
    load8(cs + half + 8 * i, n);
    uint32_t oa[4], ob[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float x0, y0, x1, y1;
      turn(bf(a[k] & 0xffffu), bf(b[k] & 0xffffu), c[2 * k], n[2 * k], x0, y0);
      turn(bf(a[k] >> 16), bf(b[k] >> 16), c[2 * k + 1], n[2 * k + 1], x1, y1);
      oa[k] = pack2(x0, x1);
      ob[k] = pack2(y0, y1);
    }
    d4[i] = make_uint4(oa[0], oa[1], oa[2], oa[3]);
    d4[i + rot / 16] = make_uint4(ob[0], ob[1], ob[2], ob[3]);
  }
};

template <int D, int GS>
__global__ void __launch_bounds__(kThreads) rotate_rows(RotateParams p) {
  constexpr int NS = D / kGroup, SPG = GS / kGroup, NG = D / GS;
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
  const RowTurn<D> rt{a.cos_sin + size_t(pos) * a.rot, a.rot, a.interleaved};
  const int per = rt.tasks();
  const int nk = lead < 0 ? 0 : p.H * per, nq = a.Q ? a.H_q * per : 0;
  for (int i = tid; i < nk + nq; i += kThreads) {
    const bool key = i < nk;
    const int j = key ? i : i - nk, head = j / per, task = j - head * per;
    if (key) {
      rt.run(a.K + (tok * p.H + head) * D, p.Kr + (size_t(row) * p.H + head) * D, task);
    } else {
      const size_t q = (tok * a.H_q + head) * D;
      rt.run(a.Q + q, a.Q_out + q, task);
    }
  }
  if (lead < 0) return;
  // ---- values: one thread per 32-channel sub-group (a group's sub-groups in
  // consecutive lanes; every lane takes part in the shuffles)
  for (int i0 = warp * 32; i0 < p.H * NS; i0 += kThreads) {
    const int i = i0 + lane;
    const bool live = i < p.H * NS;
    const int head = live ? i / NS : 0, sg = i % NS;
    uint32_t w0, w1;
    const GroupParams gp = code_values<GS>(a.V + (tok * p.H + head) * D + sg * kGroup, w0, w1);
    if (live) {
      const size_t at = (size_t(lead) * p.H + head) * size_t(p.table ? p.page : p.cap) + off;
      *reinterpret_cast<uint2*>(p.v_code + at * (D / 16) + sg * 2) = make_uint2(w0, w1);
      if (sg % SPG == 0) p.v_sz[at * NG + sg / SPG] = uint32_t(gp.s_bits) | (uint32_t(gp.z_bits) << 16);
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
  return launch_quantize(k, s);
}

}  // namespace kv2
