// Chunked prefill with sinks on tcgen05 (kvq_sinks_tc.cuh): one CTA a unit, and the choice between that and clusters.
#include "kvq_sinks_tc.cuh"

namespace kvq {
namespace {

// SMs of the current device, and how many clusters of 2, 4 and 8 CTAs run on it at once (they take the same
// shared memory and threads whatever the format).
struct Room {
  int sms, clusters[4];
};

cudaError_t room_of_device(const CacheView& v, Room* room) {
  static std::mutex mu;
  static std::map<int, Room> done;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lk(mu);
  auto it = done.find(dev);
  if (it == done.end()) {
    Room r{};
    if ((e = cudaDeviceGetAttribute(&r.sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    for (int c = 1; c < 4; ++c)
      if ((e = sinks_tc_clusters(v, r.sms >> c << c, c, &r.clusters[c])) != cudaSuccess) return e;
    it = done.emplace(dev, r).first;
  }
  *room = it->second;
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_sinks_tc(const DecodeArgs& a, cudaStream_t s) {
  Room room;
  const cudaError_t e = room_of_device(a.c, &room);
  if (e != cudaSuccess) return e;
  const int rows = (a.c.q_bits == 32 ? kQ : 2 * kQ) / a.G;
  const int units = (a.B + rows - 1) / rows * a.c.H;
  // The largest cluster of which all units' run at once (one CTA an SM: its shared memory and all of its tensor
  // memory), of 4 tiles a CTA at least
  const long long reach = (long long)a.sinks + a.span + rows, held = (long long)a.mbps * kBlock;
  const long long tiles = (reach < held ? reach : held) / kTok;
  int c = 3;
  while (c > 0 && (units > room.clusters[c] || tiles < (4 << c))) --c;
  if (c > 0) return launch_sinks_tc_shared(a, units, rows, c, s);
  return by_format<false>(a.c, [&](auto k) {
    const cudaError_t p = k.prepare();
    return p != cudaSuccess ? p : k.launch(a, units, rows, units < room.sms ? units : room.sms, 0, s);
  });
}

}  // namespace kvq
