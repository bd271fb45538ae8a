// The shared prefix of kvq_decode_shared on 16-vector query tiles.
//
// The query vectors of all sequences of a group meet the same prefix blocks: 16
// of them (rows x query heads of one KV head) are one row tile of m16n8k16, and a
// CTA streams its share of the prefix once for the tile, as the chunked prefill
// does (kvq_tiles.cuh).  The prefix of a unit is cut over several CTAs; each
// writes one record (m, l, o) per vector, and kvq_shared.cu merges the records
// with those of the suffixes.  Every cache format and query mode.  Every CTA converts each block for its 16
// vectors, so the time grows with the vectors: prefixes of 8192 tokens, int8, take 37 us a call with 16
// vectors and 46 with 64, where tcgen05 units take over (kvq_shared_tc.cu); 4 sequences on 2048 tokens: 22 us,
// latency of three launches.
#include "kvq_shared.cuh"
#include "kvq_tiles.cuh"

namespace kvq {
namespace {

template <int KB, int VB, bool ASYM, bool LOQ>
__global__ void __launch_bounds__(kThreads, 3) shared_tile_kernel(const SharedArgs sa) {
  using F = Fmt<KB, VB, ASYM>;
  using T = TileFmt<KB, VB, ASYM>;
  constexpr int S = T::kStages;
  constexpr int kStep = T::kBlocksPerStage;
  const DecodeArgs& a = sa.d;
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
  float* co = reinterpret_cast<float*>(smem);  // over the ring, once a segment has drained it
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + mp.bars);
  uint64_t* empty = full + S;
  uint64_t* cbar = empty + S;
  uint64_t* cdone = cbar + 1;
  SharedGeo* geo = reinterpret_cast<SharedGeo*>(smem + mp.total);

  const int G = a.G, H = a.c.H;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], kConsumerWarps);
    }
    mbar_init(cbar, kConsumers);
    mbar_init(cdone, 1);
    fence_mbar_init();
  }
  // keys under per-channel scales only: the key-scale slots hold 1.0 (never copied over)
  auto unit_key_scales = [&](int first, int stride) {
    for (int i = first; i < S * T::kBlocksPerStage * kBlock; i += stride) {
      const int st = i / (T::kBlocksPerStage * kBlock), r = i % (T::kBlocksPerStage * kBlock);
      reinterpret_cast<float*>(smem + st * T::kStageBytes + T::kOffMeta)[(r / kBlock) * F::kMF + F::kKS + r % kBlock] =
          1.f;
    }
  };
  if (!F::kBf16 && a.c.k_chan) unit_key_scales(tid, kThreads);
  // Beside the suffix kernel, see kvq_shared.cuh: the producer waits for it last.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  shared_geometry(geo, a, kTileQ, kStep, tid, kThreads, false);  // errors are reported by the suffix kernel
  const int Pe = shared_ctas(geo, sa.sl.ctas), ci = blockIdx.x;
  if (ci >= Pe) return wait_for_suffix();
  const long long x0 = (long long)ci * geo->T / Pe, x1 = (long long)(ci + 1) * geo->T / Pe;
  if (x0 >= x1) return wait_for_suffix();

  if (warp == kConsumerWarps) {
    // ---------------------------------------------------------------- producer
    const uint64_t pol = l2_evict_normal_policy();  // the other tiles of the group read the same blocks
    int s = 0, it = 0, seg = 0;
    uint32_t ph = 0;
    bool ok = true;
    const uint32_t meta_bytes = a.c.k_chan ? F::kMB / 2 : F::kMB;
    for (long long x = x0; x < x1 && ok; ++seg) {
      const SharedUnit un = unit_at(geo, a.num_groups, H, kStep, x);
      const long long end = min(x1, un.start + un.steps);
      const int nblk = geo->g.blocks[un.group];
      const int* table = a.table + size_t(geo->g.start[un.group]) * a.mbps;
      if (seg > 0) {  // the previous segment's merge uses the ring
        bool w_ok = true;
        if (lane == 0) w_ok = mbar_wait(cdone, uint32_t(seg - 1) & 1u);
        if (!__shfl_sync(kFull, w_ok ? 1 : 0, 0)) {
          if (lane == 0) flag(a.err, KVQ_DEVERR_TIMEOUT);
          break;
        }
      }
      for (; x < end; ++x) {
        const int b0 = int(x - un.start) * kStep, nb = min(kStep, nblk - b0);
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
          phys = __ldcg(table + b0 + lane);
          if (phys < 0 || phys >= a.c.num_blocks) {
            flag(a.err, KVQ_DEVERR_BLOCK_ID);
            phys = 0;
          }
        }
        if (lane == 0) mbar_arrive_expect_tx(&full[s], uint32_t(nb) * (F::kKBB + F::kVBB + meta_bytes));
        __syncwarp();
        if (lane < nb) {
          uint8_t* stg = smem + s * T::kStageBytes;
          const size_t hb = size_t(un.h) * a.c.num_blocks + phys;
          bulk_g2s(stg + T::kOffK + lane * F::kKBB, a.c.k_codes + hb * F::kKBB, F::kKBB, &full[s], pol);
          bulk_g2s(stg + T::kOffV + lane * F::kVBB, a.c.v_codes + hb * F::kVBB, F::kVBB, &full[s], pol);
          if constexpr (!F::kBf16) {
            if (a.c.k_chan)
              bulk_g2s(stg + T::kOffMeta + lane * F::kMB + F::kVS * 4, a.c.meta + hb * F::kMF + F::kVS, F::kMB / 2,
                       &full[s], pol);
            else
              bulk_g2s(stg + T::kOffMeta + lane * F::kMB, a.c.meta + hb * F::kMF, F::kMB, &full[s], pol);
          }
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
    return wait_for_suffix();
  }

  // ------------------------------------------------------------------ consumers
  const uint32_t km = magic_f16x2(a.B);
  const uint32_t c64 = 0x64646464u | (uint32_t(a.B) >> 16);  // a.B <= 4096: the constant itself
  const int g = lane >> 2, t = lane & 3;
  float* rec_m = reinterpret_cast<float*>(a.ws + sa.sl.off_m);
  float* rec_l = reinterpret_cast<float*>(a.ws + sa.sl.off_l);
  float* rec_o = reinterpret_cast<float*>(a.ws + sa.sl.off_rec);
  int s = 0;
  uint32_t ph = 0, cphase = 0;
  auto sync = [&]() {
    if (consumer_sync(cbar, cphase)) return true;
    flag(a.err, KVQ_DEVERR_TIMEOUT);
    return false;
  };
  for (long long x = x0; x < x1;) {
    const SharedUnit un = unit_at(geo, a.num_groups, H, kStep, x);
    const long long end = min(x1, un.start + un.steps);
    const int nblk = geo->g.blocks[un.group], first = geo->g.start[un.group];
    const int rows = geo->g.start[un.group + 1] - first;
    for (int v = warp; v < kTileQ; v += kConsumerWarps) {
      const int gv = un.tile * kTileQ + v, rr = gv / G, hj = gv % G;
      const bool act = rr < rows;
      const float qscale = stage_tile_vector<KB, ASYM, LOQ>(
          a, act ? a.q + (size_t(first + rr) * a.Hq + un.h * G + hj) * kHeadDim : nullptr, un.h, v, qf, qlo, qz_s, zo_s,
          lane);
      if (lane == 0) {
        qs_s[v] = act ? qscale : 0.f;
        qlen_s[v] = act ? prefix_len(a, first + rr, nblk) : 0;
      }
    }
    if (!sync()) return;
    const float qs0 = qs_s[g], qs1 = qs_s[g + 8];
    const float qz0 = ASYM ? qz_s[g] : 0.f, qz1 = ASYM ? qz_s[g + 8] : 0.f;
    const int len0 = qlen_s[g], len1 = qlen_s[g + 8];
    int maxlen = 0;
#pragma unroll
    for (int v = 0; v < kTileQ; ++v) maxlen = max(maxlen, qlen_s[v]);
    TileState st;
    st.reset();
    for (; x < end; ++x) {
      if (!mbar_wait(&full[s], ph)) {
        flag(a.err, KVQ_DEVERR_TIMEOUT);
        return;
      }
      const int blk = int(x - un.start) * kStep + warp;
      if (blk < nblk) {
        const uint8_t* stg = smem + s * T::kStageBytes;
        const float* meta = reinterpret_cast<const float*>(stg + T::kOffMeta + warp * F::kMB);
        tile_block<KB, VB, ASYM, LOQ, true>(stg + T::kOffK + warp * F::kKBB, stg + T::kOffV + warp * F::kVBB,
                                      meta + F::kKS, meta + F::kVS, ASYM ? meta + F::kKO : nullptr,
                                      ASYM ? meta + F::kVO : nullptr, blk * kBlock, maxlen, len0, len1, qs0, qs1, qz0,
                                      qz1, reinterpret_cast<const uint4*>(qf), reinterpret_cast<const uint4*>(qlo),
                                      reinterpret_cast<const float4*>(zo_s), st, lane, km, c64);
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
    if constexpr (ASYM) {
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
    if (!sync()) return;  // every warp has read its last block
    if (t == 0) {
      cm[warp * kTileQ + g] = st.m0 == kNegInf ? kNegInf : st.m0 - st.sg0;
      cm[warp * kTileQ + g + 8] = st.m1 == kNegInf ? kNegInf : st.m1 - st.sg1;
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
    if (!sync()) return;
    {
      const int v = tid >> 3, d0 = (tid & 7) * 16;  // 16 vectors x 8 slices of 16 dims
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
      const size_t at = size_t(ci + un.u) * kTileQ + v;
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
        *reinterpret_cast<float4*>(rec_o + at * kHeadDim + d0 + d) = make_float4(o[0], o[1], o[2], o[3]);
      }
      if ((tid & 7) == 0) {
        rec_m[at] = M;
        rec_l[at] = L;
      }
    }
    if (!sync()) return;
    if (!F::kBf16 && a.c.k_chan) unit_key_scales(tid, kConsumers);  // the merge wrote over them
    if (tid == 0) mbar_arrive(cdone);
  }
}

template <int KB, int VB, bool ASYM, bool LOQ>
struct SharedTileKernel {
  using T = TileFmt<KB, VB, ASYM>;
  static int smem_bytes() {
    return tile_smem(T::kStages * T::kStageBytes, T::kStages).total + int(sizeof(SharedGeo));
  }
  // CTAs of one wave on the current device.
  static int ctas() {
    static std::mutex mu;
    static std::map<int, int> done;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    std::lock_guard<std::mutex> lk(mu);
    auto it = done.find(dev);
    if (it != done.end()) return it->second;
    int sms = 0, per = 0;
    const auto k = shared_tile_kernel<KB, VB, ASYM, LOQ>;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes()) != cudaSuccess ||
        cudaFuncSetAttribute(k, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared) !=
            cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, k, kThreads, smem_bytes()) != cudaSuccess || per < 1)
      return 0;
    return done[dev] = sms * per;
  }
  static cudaError_t launch(const SharedArgs& a, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(a.sl.ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem_bytes();
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, shared_tile_kernel<KB, VB, ASYM, LOQ>, a);
  }
};

template <bool LOQ, class F>
auto by_format(const CacheView& c, F f) {
  const int kb = c.k_bits, vb = c.v_bits;
  const bool as = c.asym != 0;
  if (kb == 8 && vb == 8) return as ? f(SharedTileKernel<8, 8, true, LOQ>{}) : f(SharedTileKernel<8, 8, false, LOQ>{});
  if (kb == 4 && vb == 4) return as ? f(SharedTileKernel<4, 4, true, LOQ>{}) : f(SharedTileKernel<4, 4, false, LOQ>{});
  if (kb == 4 && vb == 8) return as ? f(SharedTileKernel<4, 8, true, LOQ>{}) : f(SharedTileKernel<4, 8, false, LOQ>{});
  if (kb == 8 && vb == 4) return as ? f(SharedTileKernel<8, 4, true, LOQ>{}) : f(SharedTileKernel<8, 4, false, LOQ>{});
  if (kb == 2 && vb == 2) return as ? f(SharedTileKernel<2, 2, true, LOQ>{}) : f(SharedTileKernel<2, 2, false, LOQ>{});
  return f(SharedTileKernel<16, 16, false, false>{});
}

}  // namespace

int shared_tiles_ctas(const CacheView& c) {
  const auto f = [](auto k) { return decltype(k)::ctas(); };
  return c.q_bits == 32 ? by_format<true>(c, f) : by_format<false>(c, f);
}

cudaError_t launch_shared_tiles(const SharedArgs& a, cudaStream_t s) {
  const auto f = [&](auto k) { return decltype(k)::launch(a, s); };
  return a.d.c.q_bits == 32 ? by_format<true>(a.d.c, f) : by_format<false>(a.d.c, f);
}

}  // namespace kvq
