// Chunked prefill attention on query tiles (kvq_prefill, tile path).
//
// [P3] "KV Cache Quantization and Per-Token Scale Placement", opening section:
// the cache is written incrementally and read repeatedly; a chunk of new
// positions of a sequence attends to the stored cache up to each position.
// Unlike decode, where one query group meets each cached block, a chunk has
// many query rows per block, so the contraction is dense: here a CTA takes a
// tile of 16 query vectors (consecutive rows of the call x the G query heads
// of one KV head) and every converted key and value block feeds a full
// 16-row tensor-core tile.
//
// Work: CTA (tile, kv head); tile = rows [TR*tile, TR*tile + TR) of the call,
// TR = 16 / G.  Rows of one tile that belong to different sequences are taken
// in turn ("sub-passes"), one per distinct sequence.  A producer warp streams
// the sequence's blocks 0 .. ceil(max len / 16) - 1 with bulk copies into an
// mbarrier ring, four blocks per stage; consumer warp w takes block w of each
// stage for all 16 query vectors and keeps its own online-softmax state; the
// four states are merged through shared memory at the end of a sub-pass.
//
// Scores: S (16 query vectors x 16 tokens) = Q (16 x 128, fp16, each row
// scaled by a power of two) . K^T (codes converted exactly to fp16; int8 codes
// keep the conversion's offset, 1152 + c, and each block's accumulators start
// at minus 1152 times the row's sums), two m16n8k16 products per 16-dim slice;
// the per-token key scale multiplies the scalar after the dot product ([P3]
// "The axis choice is a kernel decision").
// Values: O (16 x 128) += (P * s_v) (16 x 16 tokens, fp16) . V (codes), the
// value scale folded into the weight ([P2] "Keys and values need not have
// identical error sensitivity").  Asymmetric blocks add the key zero-point
// term m'_k * sum(q) to each score and sum(p * m'_v) to each output row, as
// the decode kernel does.  In the two-part mode (q_bits 32) the query and the
// weights p * s_v are each carried as fp16 high + low parts: a second product
// per slice with the low parts, as in decode.  The cache's fragment-native block order
// (include/kvq.h) gives each lane exactly the B-operand pairs of these
// products, the same registers the decode kernel uses as A operands.
#include "kvq_tiles.cuh"

namespace kvq {
namespace {

// A sub-pass: the rows of the tile that belong to sequence seq; nblk blocks
// cover the longest of them (maxlen tokens).
struct SubPass {
  int seq, maxlen, nblk;
};

// The sub-pass led by tile row ri (the first row of its sequence in the tile),
// or seq = -1 when row ri leads none.
__device__ __forceinline__ SubPass sub_pass_at(const int* rowseq, const int* rowlen, int nrows, int ri) {
  SubPass sp{-1, 0, 0};
  const int sb = rowseq[ri];
  if (sb < 0) return sp;
  for (int k = 0; k < ri; ++k)
    if (rowseq[k] == sb) return sp;
  int ml = 0;
  for (int k = ri; k < nrows; ++k)
    if (rowseq[k] == sb) ml = max(ml, rowlen[k]);
  sp.seq = sb;
  sp.maxlen = ml;
  sp.nblk = (ml + kBlock - 1) / kBlock;
  return sp;
}

template <int KB, int VB, bool ASYM, bool LOQ>
__global__ void __launch_bounds__(kThreads, 3) prefill_tile_kernel(const DecodeArgs a, int n_tiles, int TR) {
  using F = Fmt<KB, VB, ASYM>;
  using T = TileFmt<KB, VB, ASYM>;
  constexpr int S = T::kStages;
  extern __shared__ __align__(128) uint8_t smem[];
  const TileSmem mp = tile_smem(S * T::kStageBytes, S);
  uint32_t* qf = reinterpret_cast<uint32_t*>(smem + mp.qf);
  uint32_t* qlo = reinterpret_cast<uint32_t*>(smem + mp.qlo);
  float* qs_s = reinterpret_cast<float*>(smem + mp.qs);
  float* qz_s = reinterpret_cast<float*>(smem + mp.qz);
  float* zo_s = reinterpret_cast<float*>(smem + mp.zo);
  int* qlen_s = reinterpret_cast<int*>(smem + mp.qlen);
  float* cm = reinterpret_cast<float*>(smem + mp.cm);
  float* cl = reinterpret_cast<float*>(smem + mp.cl);
  float* co = reinterpret_cast<float*>(smem);  // over the ring (see cdone)
  int* rowseq = reinterpret_cast<int*>(smem + mp.rowseq);
  int* rowlen = reinterpret_cast<int*>(smem + mp.rowlen);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + mp.bars);
  uint64_t* empty = full + S;
  uint64_t* cbar = empty + S;
  uint64_t* cdone = cbar + 1;  // consumers have merged a sub-pass: the ring may be refilled

  const int G = a.G;
  const int tile = blockIdx.x % n_tiles, h = blockIdx.x / n_tiles;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r0 = tile * TR;
  const int nrows = min(TR, a.B - r0);

  if (tid == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], kConsumerWarps);
    }
    mbar_init(cbar, kConsumers);
    mbar_init(cdone, 1);
    fence_mbar_init();
  }
  // keys under per-channel scales only: the key-scale slots of the ring hold
  // 1.0 (the producer never copies over them; refilled after each merge)
  auto unit_key_scales = [&](int first, int stride) {
    for (int i = first; i < S * T::kBlocksPerStage * kBlock; i += stride) {
      const int st = i / (T::kBlocksPerStage * kBlock), r = i % (T::kBlocksPerStage * kBlock);
      reinterpret_cast<float*>(smem + st * T::kStageBytes + T::kOffMeta)[(r / kBlock) * F::kMF + F::kKS + r % kBlock] =
          1.f;
    }
  };
  if (a.c.k_chan) unit_key_scales(tid, kThreads);
  // programmatic dependent launch: wait for the previous kernel (the chunk's
  // quantizing write) before reading memory
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // the tile's rows: sequence and causal length (positions 0..pos), clamped to
  // the block table's capacity as kvq_decode clamps lengths; a row with an
  // invalid sequence or no position to attend to is empty (sequence -1)
  if (warp == 0 && lane < kTileQ) {
    int sb = -1, len = 0;
    if (lane < nrows) {
      sb = a.seq_of[r0 + lane];
      if (sb < 0 || sb >= a.nseq) {
        if (h == 0) flag(a.err, KVQ_DEVERR_POSITION);
        sb = -1;
      } else {
        len = a.pos[r0 + lane] + 1;
        if (len < 0 || len > table_tokens(a.mbps, 0)) {
          if (h == 0) flag(a.err, KVQ_DEVERR_SEQ_LEN);
          len = len < 0 ? 0 : table_tokens(a.mbps, 0);
        }
        if (len == 0) sb = -1;
      }
    }
    rowseq[lane] = sb;
    rowlen[lane] = len;
  }
  __syncthreads();
  // empty rows: out = 0, lse = -inf (as kvq_decode for a sequence of length 0)
  if (warp < kConsumerWarps)
    for (int i = tid; i < nrows * G * kHeadDim; i += kConsumers) {
      const int rr = i / (G * kHeadDim);
      if (rowseq[rr] >= 0) continue;
      const int hj = (i / kHeadDim) % G, d = i % kHeadDim;
      const size_t row = size_t(r0 + rr) * a.Hq + h * G + hj;
      if (a.out_fp32) reinterpret_cast<float*>(a.out)[row * kHeadDim + d] = 0.f;
      else reinterpret_cast<__nv_bfloat16*>(a.out)[row * kHeadDim + d] = __float2bfloat16_rn(0.f);
      if (d == 0 && a.lse) a.lse[row] = kNegInf;
    }

  if (warp == kConsumerWarps) {
    // ---------------------------------------------------------------- producer
    const uint64_t pol = l2_evict_normal_policy();
    int s = 0, it = 0;
    uint32_t ph = 0;
    bool ok = true;
    const uint32_t meta_bytes = a.c.k_chan ? F::kMB / 2 : F::kMB;
    int spi = 0;  // sub-passes issued
    for (int ri = 0; ri < nrows && ok; ++ri) {
      const SubPass sp = sub_pass_at(rowseq, rowlen, nrows, ri);
      if (sp.seq < 0) continue;
      if (spi > 0) {  // the previous sub-pass's merge uses the ring
        bool w_ok = true;
        if (lane == 0) w_ok = mbar_wait(cdone, uint32_t(spi - 1) & 1u);
        if (!__shfl_sync(kFull, w_ok ? 1 : 0, 0)) {
          if (lane == 0) flag(a.err, KVQ_DEVERR_TIMEOUT);
          break;
        }
      }
      ++spi;
      for (int b0 = 0; b0 < sp.nblk; b0 += T::kBlocksPerStage) {
        const int nb = min(T::kBlocksPerStage, sp.nblk - b0);
        if (it >= S) {
          bool w_ok = true;
          if (lane == 0) w_ok = mbar_wait(&empty[s], ph ^ 1u);
          if (!__shfl_sync(kFull, w_ok ? 1 : 0, 0)) {
            if (lane == 0) flag(a.err, KVQ_DEVERR_TIMEOUT);
            ok = false;
            break;
          }
        }
        int phys = 0;
        if (lane < nb) {
          phys = a.table[size_t(sp.seq) * a.mbps + b0 + lane];
          if (phys < 0 || phys >= a.c.num_blocks) {
            flag(a.err, KVQ_DEVERR_BLOCK_ID);
            phys = 0;
          }
        }
        if (lane == 0) mbar_arrive_expect_tx(&full[s], uint32_t(nb) * (F::kKBB + F::kVBB + meta_bytes));
        __syncwarp();
        if (lane < nb) {
          uint8_t* stg = smem + s * T::kStageBytes;
          const size_t hb = size_t(h) * a.c.num_blocks + phys;  // head-major pools
          bulk_g2s(stg + T::kOffK + lane * F::kKBB, a.c.k_codes + hb * F::kKBB, F::kKBB, &full[s], pol);
          bulk_g2s(stg + T::kOffV + lane * F::kVBB, a.c.v_codes + hb * F::kVBB, F::kVBB, &full[s], pol);
          if (a.c.k_chan)
            bulk_g2s(stg + T::kOffMeta + lane * F::kMB + F::kVS * 4, a.c.meta + hb * F::kMF + F::kVS, F::kMB / 2,
                     &full[s], pol);
          else
            bulk_g2s(stg + T::kOffMeta + lane * F::kMB, a.c.meta + hb * F::kMF, F::kMB, &full[s], pol);
        }
        ++it;
        if (++s == S) {
          s = 0;
          ph ^= 1u;
        }
      }
    }
    // drain: the most recent use of every stage must have landed before exit
    if (lane == 0)
      for (int k = max(0, it - S); k < it; ++k)
        if (!mbar_wait(&full[k % S], (k / S) & 1)) flag(a.err, KVQ_DEVERR_TIMEOUT);
    return;
  }

  // ------------------------------------------------------------------ consumers
  const uint32_t km = magic_f16x2(a.B);
  const uint32_t c64 = 0x64646464u | (uint32_t(a.B) >> 16);  // a.B <= 4096: the constant itself
  const int g = lane >> 2, t = lane & 3;
  const int nq = TR * G;  // query vectors of a full tile (<= 16)
  int s = 0;
  uint32_t ph = 0, cphase = 0;
  for (int ri = 0; ri < nrows; ++ri) {
    const SubPass sp = sub_pass_at(rowseq, rowlen, nrows, ri);
    if (sp.seq < 0) continue;
    // stage the sub-pass's query vectors: v = row * G + head, fp16 scaled by a
    // power of two per vector (the decode kernel's query format)
    for (int v = warp; v < kTileQ; v += kConsumerWarps) {
      const int rr = v / G, hj = v % G;
      const bool act = v < nq && rr < nrows && rowseq[rr] == sp.seq;
      const float qscale = stage_tile_vector<KB, ASYM, LOQ>(
          a, act ? a.q + (size_t(r0 + rr) * a.Hq + h * G + hj) * kHeadDim : nullptr, h, v, qf, qlo, qz_s, zo_s, lane);
      if (lane == 0) {
        qs_s[v] = act ? qscale : 0.f;
        qlen_s[v] = act ? rowlen[rr] : 0;
      }
    }
    if (!consumer_sync(cbar, cphase)) {
      flag(a.err, KVQ_DEVERR_TIMEOUT);
      return;
    }
    const float qs0 = qs_s[g], qs1 = qs_s[g + 8];
    const float qz0 = ASYM ? qz_s[g] : 0.f, qz1 = ASYM ? qz_s[g + 8] : 0.f;
    const int len0 = qlen_s[g], len1 = qlen_s[g + 8];
    TileState st;
    st.reset();
    for (int b0 = 0; b0 < sp.nblk; b0 += T::kBlocksPerStage) {
      if (!mbar_wait(&full[s], ph)) {
        flag(a.err, KVQ_DEVERR_TIMEOUT);
        return;
      }
      const int blk = b0 + warp;
      if (blk < sp.nblk) {
        const uint8_t* stg = smem + s * T::kStageBytes;
        const float* meta = reinterpret_cast<const float*>(stg + T::kOffMeta + warp * F::kMB);
        tile_block<KB, VB, ASYM, LOQ, false>(stg + T::kOffK + warp * F::kKBB, stg + T::kOffV + warp * F::kVBB,
                                      meta + F::kKS, meta + F::kVS, ASYM ? meta + F::kKO : nullptr,
                                      ASYM ? meta + F::kVO : nullptr, blk * kBlock, sp.maxlen, len0, len1, qs0, qs1,
                                      qz0, qz1, reinterpret_cast<const uint4*>(qf),
                                      reinterpret_cast<const uint4*>(qlo), reinterpret_cast<const float4*>(zo_s), st,
                                      lane, km, c64);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[s]);
      if (++s == S) {
        s = 0;
        ph ^= 1u;
      }
    }
    // ---- merge the four warps' states through shared memory
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      st.l0 += __shfl_xor_sync(kFull, st.l0, o);
      st.l1 += __shfl_xor_sync(kFull, st.l1, o);
    }
    if constexpr (ASYM) {  // the value zero-point term is the same for every output dimension
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        st.z0 += __shfl_xor_sync(kFull, st.z0, o);
        st.z1 += __shfl_xor_sync(kFull, st.z1, o);
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        st.O[i][0] += st.z0;
        st.O[i][1] += st.z0;
        st.O[i][2] += st.z1;
        st.O[i][3] += st.z1;
      }
    }
    // every warp has read its last block: the ring is free for the merge
    if (!consumer_sync(cbar, cphase)) {
      flag(a.err, KVQ_DEVERR_TIMEOUT);
      return;
    }
    if (t == 0) {
      cm[warp * kTileQ + g] = st.m0 == kNegInf ? kNegInf : st.m0 - st.sg0;
      cm[warp * kTileQ + g + 8] = st.m1 == kNegInf ? kNegInf : st.m1 - st.sg0;
      cl[warp * kTileQ + g] = st.l0;
      cl[warp * kTileQ + g + 8] = st.l1;
    }
    {
      float* ow = co + warp * kTileQ * kOStride;
#pragma unroll
      for (int nt = 0; nt < 16; ++nt) {
        *reinterpret_cast<float2*>(ow + g * kOStride + 8 * nt + 2 * t) = make_float2(st.O[nt][0], st.O[nt][1]);
        *reinterpret_cast<float2*>(ow + (g + 8) * kOStride + 8 * nt + 2 * t) = make_float2(st.O[nt][2], st.O[nt][3]);
      }
    }
    if (!consumer_sync(cbar, cphase)) {
      flag(a.err, KVQ_DEVERR_TIMEOUT);
      return;
    }
    {
      const int v = tid >> 3, d0 = (tid & 7) * 16;  // 16 vectors x 8 slices of 16 dims
      if (qlen_s[v] > 0) {
        float M = kNegInf;
#pragma unroll
        for (int w = 0; w < kConsumerWarps; ++w) M = fmaxf(M, cm[w * kTileQ + v]);
        float aw[kConsumerWarps], L = 0.f;
#pragma unroll
        for (int w = 0; w < kConsumerWarps; ++w) {
          const float mw = cm[w * kTileQ + v];
          aw[w] = (mw == kNegInf) ? 0.f : exp2f(mw - M);
          L += aw[w] * cl[w * kTileQ + v];
        }
        const float inv = 1.f / L;
        const int rr = v / G, hj = v % G;
        const size_t row = size_t(r0 + rr) * a.Hq + h * G + hj;
#pragma unroll
        for (int d = 0; d < 16; d += 4) {
          float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int w = 0; w < kConsumerWarps; ++w) {
            const float4 c = *reinterpret_cast<const float4*>(co + (w * kTileQ + v) * kOStride + d0 + d);
            o[0] = fmaf(aw[w], c.x, o[0]);
            o[1] = fmaf(aw[w], c.y, o[1]);
            o[2] = fmaf(aw[w], c.z, o[2]);
            o[3] = fmaf(aw[w], c.w, o[3]);
          }
          const size_t idx = row * kHeadDim + d0 + d;
          if (a.out_fp32) {
            *reinterpret_cast<float4*>(reinterpret_cast<float*>(a.out) + idx) =
                make_float4(o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv);
          } else {
            uint2 pk;
            pk.x = pack_bf162(o[0] * inv, o[1] * inv);
            pk.y = pack_bf162(o[2] * inv, o[3] * inv);
            *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(a.out) + idx) = pk;
          }
        }
        if ((tid & 7) == 0 && a.lse) a.lse[row] = (M + log2f(L)) * kLn2;
      }
    }
    // the next sub-pass rewrites the query tile and the combine buffers; the
    // producer may refill the ring
    if (!consumer_sync(cbar, cphase)) {
      flag(a.err, KVQ_DEVERR_TIMEOUT);
      return;
    }
    if (a.c.k_chan) unit_key_scales(tid, kConsumers);  // the merge wrote over them
    if (tid == 0) mbar_arrive(cdone);
  }
}

template <int KB, int VB, bool ASYM, bool LOQ>
struct TileKernel {
  using T = TileFmt<KB, VB, ASYM>;
  static int smem_bytes() { return tile_smem(T::kStages * T::kStageBytes, T::kStages).total; }
  static cudaError_t launch(const DecodeArgs& a, cudaStream_t s) {
    static std::mutex mu;
    static std::map<int, bool> done;
    int dev = 0;
    cudaGetDevice(&dev);
    {
      std::lock_guard<std::mutex> lk(mu);
      if (!done.count(dev)) {
        cudaFuncSetAttribute(prefill_tile_kernel<KB, VB, ASYM, LOQ>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes());
        cudaFuncSetAttribute(prefill_tile_kernel<KB, VB, ASYM, LOQ>, cudaFuncAttributePreferredSharedMemoryCarveout,
                             cudaSharedmemCarveoutMaxShared);
        done[dev] = true;
      }
    }
    const int TR = kTileQ / a.G;
    const int n_tiles = (a.B + TR - 1) / TR;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(n_tiles * a.c.H));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem_bytes();
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, prefill_tile_kernel<KB, VB, ASYM, LOQ>, a, n_tiles, TR);
  }
};

}  // namespace

bool prefill_tiles_supported(const CacheView& c) {
  const bool bits = ((c.k_bits == 8 || c.k_bits == 4) && (c.v_bits == 8 || c.v_bits == 4)) ||
                    (c.k_bits == 2 && c.v_bits == 2);
  return bits && (c.q_bits == 0 || c.q_bits == 16 || c.q_bits == 8 || c.q_bits == 32) && c.window == 0;
}

template <bool ASYM, bool LOQ>
cudaError_t launch_tiles(const DecodeArgs& a, cudaStream_t s) {
  if (a.c.k_bits == 8 && a.c.v_bits == 8) return TileKernel<8, 8, ASYM, LOQ>::launch(a, s);
  if (a.c.k_bits == 4 && a.c.v_bits == 4) return TileKernel<4, 4, ASYM, LOQ>::launch(a, s);
  if (a.c.k_bits == 4 && a.c.v_bits == 8) return TileKernel<4, 8, ASYM, LOQ>::launch(a, s);
  if (a.c.k_bits == 8 && a.c.v_bits == 4) return TileKernel<8, 4, ASYM, LOQ>::launch(a, s);
  if (a.c.k_bits == 2 && a.c.v_bits == 2) return TileKernel<2, 2, ASYM, LOQ>::launch(a, s);
  return cudaErrorInvalidValue;
}

cudaError_t launch_prefill_tiles(const DecodeArgs& a, cudaStream_t s) {
  const bool loq = a.c.q_bits == 32;
  if (a.c.asym) return loq ? launch_tiles<true, true>(a, s) : launch_tiles<true, false>(a, s);
  return loq ? launch_tiles<false, true>(a, s) : launch_tiles<false, false>(a, s);
}

}  // namespace kvq
