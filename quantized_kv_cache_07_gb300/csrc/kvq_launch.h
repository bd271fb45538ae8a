// Internal host-side interface between the C ABI (kvq_api.cu) and the kernel
// translation units.  Not part of the public ABI.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace kvq {

struct CacheView {
  int H;            // KV heads
  int num_blocks;
  int k_bits, v_bits;
  uint8_t* k_codes;
  uint8_t* v_codes;
  float* meta;      // [H][num_blocks][meta_floats]: K scales, (K zero points,) V scales, (V zero points)
  int asym;         // 1: scale and zero point per token (meta_floats 64), else 32
  int meta_floats;
  const float* factor;  // [H][128] or null
  int window, window_batch;
  int q_bits;      // query format: 8 int8 rows (integer dot), 16 fp16, 32 fp16 hi + lo
  int k_chan;      // 1: keys carry per-channel scales (factor) only, no per-token key scale
  uint8_t* k_win;  // bf16 ring: [window_batch][H][W/16] fragment-native bf16 blocks
  uint8_t* v_win;
};

struct AppendArgs {
  CacheView c;
  const uint16_t* k_new;
  const uint16_t* v_new;
  int n;
  const int* seq_idx;
  const int* pos;
  int mode;
  const int* table;
  int batch;
  int mbps;
  uint32_t* err;
};

// Rotary write: the append arguments (k_new, v_new with row strides in elements)
// plus queries and the table of cosines and sines.
struct RopeArgs {
  AppendArgs ap;
  bool write;  // keys and values given
  const uint16_t* q;
  uint16_t* q_out;
  int Hq;  // query heads to turn (0: none)
  long long q_stride, k_stride, v_stride;
  const float* table;  // [max_pos][R / 2][2]
  int R, max_pos;
  bool interleaved;
  const int* rope_pos;
};

struct RopeFreqs {
  double f[64];
  double amplitude;
};

struct MassArgs {
  CacheView c;
  const uint16_t* q;  // bf16 [B][Hq][128]
  int B, Hq, G;
  const float* lse;  // [B][Hq]
  const int* seq_lens;
  const int* table;
  int mbps;
  float* mass;  // [B][H][stride]
  int stride;
  float decay;
  uint32_t* err;
};

constexpr int kMaxBatch = 4096;  // sequence geometry is staged in shared memory

struct EvictArgs {
  CacheView c;
  const float* mass;  // [B][H][stride], as all per-token rows
  float* mass_out;    // or null
  const int* token_pos;  // or null: the slot
  int* pos_out;          // or null
  const int* next_pos;   // [B] or null: the length
  int* source;
  int* new_lens;  // [B]
  const int* seq_lens;
  const int* keep;  // [B]
  int stride, protect_first, protect_recent;
  const int* table;
  int B, mbps;
  uint32_t* err;
};

struct DequantArgs {
  CacheView c;
  const int* slots;
  int n;
  float* k_out;
  float* v_out;
  bool wide;  // outputs aligned to 16 bytes
};

// Workspace layout of a decode call (byte offsets from the workspace base).
struct DecodeLayout {
  int stream_ctas, window_ctas, units, slots;
  int switch_blocks;  // virtual blocks charged for starting a unit (0: unit-aligned split)
  size_t off_counter;  // int [units]: merge arrival counters
  size_t off_m, off_l, off_o, total;  // partial records: m, l [slots][G], o [slots][G][128]
};

struct DecodeArgs {
  CacheView c;
  const uint16_t* q;  // bf16 [B][Hq][128]
  int B, Hq, G;
  const int* seq_lens;
  // Prefill (pos != null): row b of the call is position pos[b] of sequence
  // seq_of[b] (< nseq); it attends to positions 0..pos[b] of that sequence.
  const int* pos;
  const int* seq_of;
  int nseq;
  const int* table;
  int mbps;
  void* out;
  int out_fp32;
  float* lse;
  uint8_t* ws;
  DecodeLayout lay;
  uint32_t* err;
  // 1: seq_lens and the block table are final before the preceding kernel on
  // the stream ends (KVQ_DECODE_GEOMETRY_READY): read them before the wait
  int ahead = 0;
  // kvq_decode_shared: groups of sequences with a common prefix
  const int* group_start = nullptr;    // [num_groups + 1]
  const int* prefix_blocks = nullptr;  // [num_groups]
  int num_groups = 0;
};

constexpr int kMaxGroups = 256;

// Workspace of kvq_decode_shared (byte offsets).  The prefix is split over `ctas` CTAs; a unit is
// a tile of `unit` query vectors of one group and KV head; CTA c's share of unit u is record c + u, with room for
// `tile` vectors (twice the unit where two warpgroups leave a record each).
// The suffixes are split into chunks over `suf_ctas` CTAs, one record each, and one per unit for a
// bf16 window behind them.
struct SharedLayout {
  int ctas, tile, unit, slots;
  bool tc;  // tcgen05 path (tile 256), else mma.sync (tile 16)
  int suf_ctas, suf_slots;
  size_t off_m, off_l, off_rec;     // prefix records: float [slots][tile], twice, and [slots][tile][128]
  size_t off_sm, off_sl, off_so;    // suffix records: float [suf_slots][G], twice, and [suf_slots][G][128]
  size_t off_chunks;                // int2 [B]: first chunk of a sequence, chunks of each of its heads
  size_t total;
};

struct SharedArgs {
  DecodeArgs d;  // out, lse: the caller's
  SharedLayout sl;
};

// The largest GQA group (query heads per KV head) the decode kernel takes: one
// 8-wide MMA tile of query columns.
constexpr int kMaxGroup = 8;

// Unit-start charge of the split, in blocks of the cache's format.
int switch_blocks_for(int k_bits);
// switch_cost: the unit-start charge when the split is not unit-aligned.
DecodeLayout decode_layout(int B, int Hq, int H, int window, int stream_ctas, int switch_cost);

// Every launch gives its own status (cudaLaunchKernelEx returns it): the runtime's last error is not read, since it
// may be that of an earlier call that the caller has dealt with.
cudaError_t launch_append(const AppendArgs& a, cudaStream_t s);
cudaError_t launch_rope_append(const RopeArgs& a, cudaStream_t s);
cudaError_t launch_rope_table(const RopeFreqs& f, int pairs, int max_pos, float* table, cudaStream_t s);
cudaError_t launch_mass(const MassArgs& a, cudaStream_t s);
cudaError_t launch_evict(const EvictArgs& a, cudaStream_t s);
cudaError_t launch_dequant(const DequantArgs& a, cudaStream_t s);
// Resident decode CTAs per SM for this cache format and batch (occupancy
// query on the current device, cached); 0 for an unsupported format.
int decode_ctas_per_sm_for(int k_bits, int v_bits, bool asym, int q_bits, int batch, bool rows = false);
cudaError_t launch_decode(const DecodeArgs& a, cudaStream_t s);
// The asymmetric instantiations (kvq_decode_asym.cu).
int decode_ctas_per_sm_asym(int k_bits, int v_bits, int batch, bool rows);
cudaError_t launch_decode_asym(const DecodeArgs& a, cudaStream_t s);
// The two-part fp16 query instantiations (kvq_decode_q32.cu).
int decode_ctas_per_sm_q32(int k_bits, int v_bits, bool asym, int batch, bool rows);
cudaError_t launch_decode_q32(const DecodeArgs& a, cudaStream_t s);
// kvq_decode_shared: the suffixes (kvq_suffix*.cu), the prefix on query tiles
// (kvq_shared_tiles.cu: mma.sync, kvq_shared_tc.cu: tcgen05) and the merge (kvq_shared.cu).
// The *_ctas functions give one wave on the current device, 0 on failure.
int suffix_ctas(const CacheView& c, int batch);
cudaError_t launch_suffix(const SharedArgs& a, cudaStream_t s);
int suffix_ctas_q32(const CacheView& c, int batch);
cudaError_t launch_suffix_q32(const SharedArgs& a, cudaStream_t s);
int shared_tiles_ctas(const CacheView& c);
cudaError_t launch_shared_tiles(const SharedArgs& a, cudaStream_t s);
int shared_tc_ctas(const CacheView& c);
cudaError_t launch_shared_tc(const SharedArgs& a, cudaStream_t s);
cudaError_t launch_shared_merge(const SharedArgs& a, cudaStream_t s);
// Prefill on 16-vector query tiles (kvq_prefill_tiles.cu): quantized blocks
// (8-, 4- or 2-bit, symmetric or asymmetric), any query format, no window.
// Needs no workspace.
bool prefill_tiles_supported(const CacheView& c);
cudaError_t launch_prefill_tiles(const DecodeArgs& a, cudaStream_t s);

}  // namespace kvq
