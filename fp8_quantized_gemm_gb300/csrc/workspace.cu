// Device scratch of the calls whose interface has none: the E8M0 words that
// the UE8M0 per-group GEMMs beyond one row tile expand their scales into.
//
// Outside a stream capture, each stream has a buffer of its own (the calls of a
// stream follow one another), grown by doubling.  Streams are told apart by
// their id, which the runtime never issues twice (a handle may be issued again
// while the work of the stream that had it still runs).  A buffer outlives its
// stream, so only the first kMaxStreams streams have one; the calls on any
// others allocate and free in the stream's order, which costs them two more
// runtime calls.
//
// A captured call gets a buffer of its graph: replays may run at any time and
// on any stream, beside direct calls and other graphs, so they share memory
// with neither.  The calls that one capture records on one stream share a
// buffer, as their nodes follow one another.  The graph (and every executable
// graph made of it) holds a reference; when the last one is gone, after the
// last replay has ended, the buffer becomes free for another capture or stream.
//
// No buffer is returned to the driver: cudaFree waits for the device.
#include "workspace.h"

#include <map>
#include <mutex>
#include <tuple>
#include <vector>

namespace fp8k {
namespace {

struct Buffer {
  int dev = 0;
  void *ptr = nullptr;
  size_t bytes = 0;
};
struct Recorded {
  unsigned long long capture = 0;
  Buffer buf;
};

constexpr size_t kMaxStreams = 64;

// Never destroyed: graphs may release their buffers while the process exits.
struct State {
  std::mutex mu;  // of the two maps; held while a Workspace lives
  std::map<std::tuple<int, unsigned long long>, Buffer> kept;  // by device and stream id
  std::map<std::tuple<int, cudaStream_t>, Recorded> recorded;  // of the latest capture on each
  std::mutex free_mu;                // taken by graphs' releases too, which may make no CUDA call
  std::vector<Buffer> free;
};
State &state() {
  static State *s = new State;
  return *s;
}

void give_back(const Buffer &b) noexcept {
  if (b.ptr == nullptr) return;
  try {
    State &s = state();
    std::lock_guard<std::mutex> lk(s.free_mu);
    s.free.push_back(b);
  } catch (...) {  // no host memory for the list: the buffer stays unused
  }
}

void release(void *p) {  // of a graph's reference
  Buffer *b = static_cast<Buffer *>(p);
  give_back(*b);
  delete b;
}

// Allocates and waits even while another thread or stream is captured: these
// calls touch no capturing stream.
struct RelaxedCapture {
  cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
  RelaxedCapture() { cudaThreadExchangeStreamCaptureMode(&mode); }
  ~RelaxedCapture() { cudaThreadExchangeStreamCaptureMode(&mode); }
  RelaxedCapture(const RelaxedCapture &) = delete;
  RelaxedCapture &operator=(const RelaxedCapture &) = delete;
};

// A free buffer of at least `bytes` (the smallest), or a new one.
cudaError_t take(int dev, size_t bytes, Buffer *out) {
  State &s = state();
  {
    std::lock_guard<std::mutex> lk(s.free_mu);
    size_t best = s.free.size();
    for (size_t i = 0; i < s.free.size(); ++i)
      if (s.free[i].dev == dev && s.free[i].bytes >= bytes &&
          (best == s.free.size() || s.free[i].bytes < s.free[best].bytes))
        best = i;
    if (best < s.free.size()) {
      *out = s.free[best];
      s.free.erase(s.free.begin() + (long)best);
      return cudaSuccess;
    }
  }
  bytes = (bytes + (1u << 20) - 1) & ~(size_t)((1u << 20) - 1);
  void *p = nullptr;
  const cudaError_t e = cudaMalloc(&p, bytes);
  if (e != cudaSuccess) return e;
  out->dev = dev;
  out->ptr = p;
  out->bytes = bytes;
  return cudaSuccess;
}

// (A stream that is being captured has no id; its handle stays its own until
// the capture, named by an id that is never issued again either, has ended.)
cudaError_t for_capture(int dev, cudaStream_t st, unsigned long long capture, cudaGraph_t graph,
                        size_t need, void **out) {
  Recorded &r = state().recorded[{dev, st}];
  if (r.capture != capture || r.buf.bytes < need) {
    Buffer *owned = new Buffer;
    cudaError_t e = take(dev, need, owned);
    if (e != cudaSuccess) {
      delete owned;
      return e;
    }
    const Buffer b = *owned;
    cudaUserObject_t ref = nullptr;
    e = cudaUserObjectCreate(&ref, owned, release, 1, cudaUserObjectNoDestructorSync);
    if (e != cudaSuccess) {
      release(owned);
      return e;
    }
    e = cudaGraphRetainUserObject(graph, ref, 1, cudaGraphUserObjectMove);
    if (e != cudaSuccess) {
      cudaUserObjectRelease(ref, 1);
      return e;
    }
    r.capture = capture;
    r.buf = b;
  }
  *out = r.buf.ptr;
  return cudaSuccess;
}

cudaError_t for_stream(Buffer &w, int dev, cudaStream_t st, size_t need, void **out) {
  if (w.bytes < need) {
    Buffer b;
    cudaError_t e = take(dev, need > 2 * w.bytes ? need : 2 * w.bytes, &b);
    if (e != cudaSuccess) return e;
    if (w.ptr != nullptr && (e = cudaStreamSynchronize(st)) != cudaSuccess) {
      give_back(b);
      return e;
    }
    give_back(w);
    w = b;
  }
  *out = w.ptr;
  return cudaSuccess;
}

}  // namespace

cudaError_t Workspace::get(cudaStream_t st, size_t need) {
  try {  // the callers are C functions
    return find(st, need);
  } catch (...) {
    return cudaErrorMemoryAllocation;
  }
}

cudaError_t Workspace::find(cudaStream_t st, size_t need) {
  int dev = 0;
  unsigned long long id = 0, capture = 0;
  cudaStreamCaptureStatus status = cudaStreamCaptureStatusNone;
  cudaGraph_t graph = nullptr;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess)
    e = cudaStreamGetCaptureInfo(st, &status, &capture, &graph, nullptr, nullptr, nullptr);
  if (e != cudaSuccess) return e;
  if (status == cudaStreamCaptureStatusInvalidated) return cudaErrorStreamCaptureInvalidated;
  State &s = state();
  lock_ = std::unique_lock<std::mutex>(s.mu);
  const RelaxedCapture relaxed;
  if (status == cudaStreamCaptureStatusActive)
    return for_capture(dev, st, capture, graph, need, &ptr_);
  if ((e = cudaStreamGetId(st, &id)) != cudaSuccess) return e;
  const std::tuple<int, unsigned long long> key(dev, id);
  auto at = s.kept.find(key);
  if (at == s.kept.end() && s.kept.size() < kMaxStreams) at = s.kept.emplace(key, Buffer{}).first;
  if (at != s.kept.end()) return for_stream(at->second, dev, st, need, &ptr_);
  if ((e = cudaMallocAsync(&ptr_, need, st)) != cudaSuccess) return e;
  st_ = st;
  ordered_ = true;
  return cudaSuccess;
}

Workspace::~Workspace() {
  if (ordered_) cudaFreeAsync(ptr_, st_);
}

}  // namespace fp8k
