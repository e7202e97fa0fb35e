// Internal declarations shared by the host entry points and the kernel files
// of libkv2. Nothing here is part of the C ABI (see include/kv2.h).
#pragma once

#include <cstddef>
#include <cstdint>
#include <climits>

#include <cuda_runtime.h>

#include "kv2.h"

namespace kv2 {

constexpr int kGroup = 32;          // channels of a sub-group: one code-word pair, one 8-bit q.k k-step
constexpr int kMaxCentroids = 512;  // centroid ids fit in u16 above 256

// Channels per (scale, zero) group of a cache descriptor (0 selects 32).
inline int cache_group(const kv2_cache& c) { return c.group ? c.group : kGroup; }

// Arguments of one quantize/append call (validated by the host entry point).
struct QuantizeArgs {
  const uint16_t* K;   // bf16 [B][n_new][H][d]
  const uint16_t* V;
  int B, H, d, M, r, cap, n_new, pos, C;
  const uint16_t* cent;  // fp16 [H][M][d]
  const float* P;        // [H][d][r]
  const float* w;        // [H][d]
  const float* Wg;       // [H][d/group]
  uint32_t* k_code;
  uint32_t* v_code;
  uint32_t* k_sz;
  uint32_t* v_sz;
  void* cidx;
  uint16_t* psac;
  // assignment only (centre fitting): when set, the chosen centre of row
  // (b * n_new + t) and head h goes to assign[row * H + h] and nothing is
  // packed (V, P and the cache streams are not read or written)
  int32_t* assign = nullptr;
  // PSAC storage: 0 = fp16 coefficients in psac; 1 = int8 codes in psac and
  // one fp16 scale per token in psac_scale
  int psac_fmt = 0;
  uint16_t* psac_scale = nullptr;
  // paged cache: block table [B][cap / page] (null: contiguous streams)
  const int32_t* table = nullptr;
  int page = 0;
  int group = kGroup;  // channels per (scale, zero) group: 32, 64 or 128
  // rows with places of their own, written by the kernel just before on the
  // stream (the key kernel is then its programmatic dependent): row i of K
  // [*n_rows][H][d] goes to offset rows[i].y of sequence or page rows[i].x
  // (negative: not stored); B * n_new bounds their number; V null: values are
  // coded elsewhere
  const int2* rows = nullptr;
  const int* n_rows = nullptr;
};
cudaError_t launch_quantize(const QuantizeArgs& a, cudaStream_t s);
cudaError_t launch_quantize_rows(const QuantizeArgs& a, cudaStream_t s);   // a.rows, a.n_rows

// Append with the position rotation applied on the way, at per-sequence places.
struct RotaryArgs {
  const kv2_cache* c;
  const float* cos_sin;      // [positions][rot]: rot/2 cosines, rot/2 sines
  int positions, rot, interleaved;
  const uint16_t* K;         // bf16 [B][n_new][H_kv][d]
  const uint16_t* V;
  const uint16_t* Q;         // bf16 [B][n_new][H_q][d] (null: no queries)
  uint16_t* Q_out;
  int H_q;
  const int32_t* position;   // [B][n_new]
  const int32_t* start;      // [B]
  const int32_t* count;      // [B] (null: n_new each)
  int n_new, candidates;
  void* ws;
};
size_t rotary_workspace_bytes(const kv2_cache& c, int n_new);
cudaError_t launch_rotary(const RotaryArgs& a, const QuantizeArgs& q, cudaStream_t s);

// QSAC-aware centre fitting (Lloyd iterations with the QSAC assignment).
struct FitCentroidsArgs {
  const uint16_t* X;   // bf16 [n][H][D] sample keys
  int n, H, D, M, C, iters;
  const float* w;      // [H][D]
  const float* Wg;     // [H][D/group]
  uint16_t* cent;      // fp16 [H][M][D], initial centres in, fitted centres out
  int32_t* assign;     // [n][H]: the last assignment
  void* ws;            // fit_centroids_workspace_bytes(H, D, M)
  int group = kGroup;  // channels per (scale, zero) group of the QSAC estimate
};
size_t fit_centroids_workspace_bytes(int H, int D, int M);

// Most-attended token per query (retrieval analysis): over the packed cache
// (c set, K null) or over dense bf16 keys K [B][len][H_kv][d] (c null).
struct Top1Args {
  const kv2_cache* c;
  const uint16_t* Q;   // bf16 [B][nq][H_q][d]
  const uint16_t* K;
  int B, nq, H_q, H_kv, d, len;
  int32_t* top1;       // [B][nq][H_q]
  void* ws;            // top1_workspace_bytes(B, nq, H_q, len)
};
size_t top1_workspace_bytes(int B, int nq, int H_q, int len);
cudaError_t launch_top1(const Top1Args& a, cudaStream_t s);
cudaError_t launch_fit_centroids(const FitCentroidsArgs& a, cudaStream_t s);

// Decode attention.
struct DecodeArgs {
  const kv2_cache* c;   // host copy of the descriptor
  int len, H_q;
  const uint16_t* Q;    // bf16 [B][H_q][d]
  float sm_scale;
  void* out;
  int out_dtype;
  void* ws;
  size_t ws_bytes;
  // Slots at or after wait_from are written by the kernel just before on the
  // stream; the decode then starts as its programmatic dependent and waits
  // for it only before copying a tile that reaches such a slot. INT32_MAX:
  // ordinary stream order.
  int wait_from = INT32_MAX;
  // cross attention and shared prefixes: lengths from `lens`, heads scaled by themselves
  bool rows = false;
  const int32_t* lens = nullptr;    // device [B]: tokens per sequence, taken into 0..len (null: len each)
  const int32_t* q_lens = nullptr;  // device [B]: sequences of no query (<= 0) are not written (null: all are)
};
size_t decode_workspace_bytes(const kv2_cache& c, int H_q, int len);
cudaError_t launch_decode(const DecodeArgs& a, cudaStream_t s);
// Its first kernel alone: per (sequence, KV head), split and query head of the
// group, d unnormalised sums, the running maximum (log2 units) and the softmax
// denominator, [B * H_kv][splits][G][d + 2].
int decode_splits(const kv2_cache& c, int H_q, int len);
cudaError_t launch_decode_split(const DecodeArgs& a, float* part, cudaStream_t s);

// PSAC basis fit.
struct FitArgs {
  const uint16_t* Qhist;  // bf16 [n][H_q][d]
  int n, H_q, H_kv, d, r;
  float* P;
  float* w;
  float* Wg;
  float* energy;
  void* ws;
  int group = kGroup;     // Wg sums w over groups of this many channels
};
size_t fit_workspace_bytes(int H_kv, int d);
cudaError_t launch_fit(const FitArgs& a, cudaStream_t s);

// Chunk attention (tcgen05).
struct ChunkArgs {
  const kv2_cache* c;
  int len, H_q, Nq, frame_tokens;
  const uint16_t* Q;      // bf16 [B][Nq][H_q][d]
  const uint16_t* Kself;  // bf16 [B][Nq][H_kv][d]
  const uint16_t* Vself;
  float sm_scale;
  void* out;
  int out_dtype;
  void* ws;
  size_t ws_bytes;
  int* err_flag;          // device word for bounded-wait timeouts (in ws)
};
size_t chunk_workspace_bytes(const kv2_cache& c, int H_q, int Nq);
cudaError_t launch_chunk(const ChunkArgs& a, cudaStream_t s);

// Rows of queries that read the same keys (tcgen05): one source (cross
// attention) or two (a shared prefix, then each sequence's own cache).
struct RowsInput {
  const kv2_cache* c;
  const int32_t* lens;    // device [B]: cached tokens per sequence (null: max_len each)
  const int32_t* q_lens;  // device [B]: queries per sequence (null: Nq each)
  int max_len, Nq;
};
struct RowsArgs {
  RowsInput src[2];
  int nsrc, H_q;
  const uint16_t* Q;      // bf16 [src[0].B][src[0].Nq][H_q][d]; the same rows for both sources
  float sm_scale;
  void* out;
  int out_dtype;
  void* ws;
};
size_t rows_workspace_bytes(const RowsArgs& a);
cudaError_t launch_rows(const RowsArgs& a, cudaStream_t s);

// Records the detail returned by kv2_last_error() on this thread; returns st.
kv2_status set_last_error(kv2_status st, const char* fmt, ...);
// Every check kv2_attention_decode makes except those of the workspace; on
// success *ws_need is the workspace size the call needs.
kv2_status validate_decode(const kv2_cache* c, int len, const uint16_t* Q, int H_q, void* out, int out_dtype,
                           size_t* ws_need);

}  // namespace kv2
