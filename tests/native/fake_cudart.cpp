// A stand-in for the CUDA runtime, for tests of the library's host side without a GPU: its
// objects are linked with this file in place of the runtime.  Nothing is ever launched.  A launch is
// written to a log (kernel, device, stream, whether it may start under the launch before it) and refused
// as the runtime refuses it when it wants more dynamic shared memory than the kernel was allowed on
// the current device.  On a stream that a test has set to capture, a launch becomes the one node that the
// stream depends on.  `fake_hook` is called inside every launch, so that a test can make
// another call there, as another host thread would.
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>
#include <map>
#include <mutex>
#include <string>
#include <utility>
#include <vector>

namespace {
struct Launch {
  std::string kernel;
  int device;
  unsigned long long stream;
  int overlaps, smem, status;
};
std::recursive_mutex mu;
std::map<const void*, std::string>& names() {
  static std::map<const void*, std::string> m;
  return m;
}
std::map<std::pair<const void*, int>, int> allowed;   // dynamic shared memory by kernel and device
std::vector<Launch> launches;
struct Capture {
  unsigned long long id;
  std::vector<cudaGraphNode_t> nodes;   // that the stream depends on
};
std::map<unsigned long long, Capture> capturing;   // by stream
uintptr_t nodes_made = 0;
thread_local int device = 0;
thread_local cudaError_t last_error = cudaSuccess;
int attribute_failures = 0, attribute_calls = 0, launch_failures = 0;
void (*hook)() = nullptr;
unsigned words[64][4];
void* handle[1];
}  // namespace

extern "C" {
void** __cudaRegisterFatBinary(void*) { return handle; }
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterFunction(void**, const char* fn, char*, const char* name, int, void*, void*, void*, void*, int*) {
  names()[fn] = name;
}
void __cudaRegisterVar(void**, char*, char*, const char*, int, size_t, int, int) {}
unsigned __cudaPopCallConfiguration(dim3*, dim3*, size_t*, void*) { return 0; }
cudaError_t __cudaGetKernel(cudaKernel_t*, const void*) { return cudaErrorNotSupported; }
cudaError_t __cudaLaunchKernel(cudaKernel_t, dim3, dim3, void**, size_t, cudaStream_t) { return cudaErrorNotSupported; }

cudaError_t cudaGetDevice(int* d) {
  *d = device;
  return cudaSuccess;
}
cudaError_t cudaGetLastError() {
  const cudaError_t e = last_error;
  last_error = cudaSuccess;
  return e;
}
const char* cudaGetErrorString(cudaError_t e) { return e == cudaErrorInvalidValue ? "invalid argument" : "error"; }
cudaError_t cudaGetSymbolAddress(void** p, const void*) {
  *p = words[device];
  return cudaSuccess;
}
cudaError_t cudaMemcpy(void* dst, const void* src, size_t n, cudaMemcpyKind) {
  std::memcpy(dst, src, n);
  return cudaSuccess;
}
cudaError_t cudaStreamSynchronize(cudaStream_t) { return cudaSuccess; }
cudaError_t cudaOccupancyMaxActiveClusters(int* n, const void*, const cudaLaunchConfig_t*) {
  *n = 64;
  return cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void* fn, cudaFuncAttribute a, int v) {
  std::lock_guard<std::recursive_mutex> lock(mu);
  ++attribute_calls;
  if (attribute_failures > 0) {
    --attribute_failures;
    return last_error = cudaErrorInvalidValue;
  }
  if (a == cudaFuncAttributeMaxDynamicSharedMemorySize) allowed[{fn, device}] = v;
  return cudaSuccess;
}
cudaError_t cudaStreamGetCaptureInfo(cudaStream_t s, cudaStreamCaptureStatus* status, unsigned long long* id,
                                     cudaGraph_t*, const cudaGraphNode_t** nodes, const cudaGraphEdgeData**,
                                     size_t* n) {
  std::lock_guard<std::recursive_mutex> lock(mu);
  const auto it = capturing.find((unsigned long long)(uintptr_t)s);
  *status = it == capturing.end() ? cudaStreamCaptureStatusNone : cudaStreamCaptureStatusActive;
  if (it == capturing.end()) return cudaSuccess;
  if (id) *id = it->second.id;
  if (nodes) *nodes = it->second.nodes.data();
  if (n) *n = it->second.nodes.size();
  return cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* fn, void**) {
  std::lock_guard<std::recursive_mutex> lock(mu);
  if (void (*h)() = hook) {
    hook = nullptr;
    h();
  }
  Launch l;
  l.kernel = names().count(fn) ? names()[fn] : "?";
  l.device = device;
  l.stream = (unsigned long long)(uintptr_t)c->stream;
  l.smem = (int)c->dynamicSmemBytes;
  l.overlaps = 0;
  for (unsigned i = 0; i < c->numAttrs; ++i)
    if (c->attrs[i].id == cudaLaunchAttributeProgrammaticStreamSerialization)
      l.overlaps = c->attrs[i].val.programmaticStreamSerializationAllowed;
  const auto a = allowed.find({fn, device});
  l.status = l.smem > 48 * 1024 && (a == allowed.end() || a->second < l.smem) ? cudaErrorInvalidValue : cudaSuccess;
  if (launch_failures > 0) {
    --launch_failures;
    l.status = cudaErrorInvalidValue;
  }
  launches.push_back(l);
  const auto cap = capturing.find(l.stream);
  if (cap != capturing.end() && !l.status) cap->second.nodes = {(cudaGraphNode_t)(16 * ++nodes_made)};
  if (l.status) last_error = (cudaError_t)l.status;
  return (cudaError_t)l.status;
}

// Tensor maps: accepted as they come.
static int encode_any(...) { return 0; }
cudaError_t cudaGetDriverEntryPointByVersion(const char*, void** p, unsigned, unsigned long long,
                                             cudaDriverEntryPointQueryResult* q) {
  *p = reinterpret_cast<void*>(encode_any);
  *q = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}

// ---- the test's side
void fake_device(int d) { device = d; }
void fake_hook(void (*h)()) { hook = h; }   // called once, inside the next launch and before it
void fake_capture(unsigned long long stream, unsigned long long id) {   // id 0: the capture ends
  if (id) capturing[stream] = {id, {}};
  else capturing.erase(stream);
}
// `stream` waits for an event that was recorded on `other`, or (other == stream) another library's kernel
void fake_join(unsigned long long stream, unsigned long long other) {
  if (stream == other) {
    capturing[stream].nodes = {(cudaGraphNode_t)(16 * ++nodes_made)};
    return;
  }
  Capture& c = capturing[stream];
  c.id = capturing[other].id;
  for (cudaGraphNode_t n : capturing[other].nodes) c.nodes.push_back(n);
}
void fake_fail_attributes(int n) { attribute_failures = n; }
void fake_fail_launches(int n) { launch_failures = n; }
int fake_attribute_calls() { return attribute_calls; }
void fake_status(unsigned v) { words[device][0] = v; }
int fake_launches() { return (int)launches.size(); }
void fake_clear() { launches.clear(); }
const char* fake_kernel(int i) { return launches[i].kernel.c_str(); }
int fake_launch(int i, unsigned long long* stream, int* dev, int* smem, int* status) {
  const Launch& l = launches[i];
  *stream = l.stream;
  *dev = l.device;
  *smem = l.smem;
  *status = l.status;
  return l.overlaps;
}
}
