// A CUDA runtime of several devices that runs nothing, for the host side of
// the training operators: linked with their objects in place of the runtime.
//
//   fake_runtime devices   parts of a backward pass on devices of 152, 76 and 10 SMs, in turn
//   fake_runtime threads   the same size asked for by 16 threads at once, while the runtime's
//                          answer changes from call to call
#include <cuda_runtime.h>

#include <atomic>
#include <cstdio>
#include <cstring>
#include <thread>
#include <vector>

#include "xp_train.h"

namespace {
constexpr int kSms[] = {152, 76, 10};
thread_local int current = 0;
std::atomic<int> asked{0};
bool changing = false;
}  // namespace

namespace xp {
void set_last_error(const char*) {}
}  // namespace xp

extern "C" {
cudaError_t cudaGetDevice(int* d) { return *d = current, cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr, int d) {
  *v = kSms[d] + (changing ? asked.fetch_add(1) : 0);
  return cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveClusters(int* n, const void*, const cudaLaunchConfig_t* c) {
  *n = kSms[current] / (2 * (int)c->gridDim.x) + (changing ? asked.fetch_add(1) : 0);
  return cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int) { return cudaSuccess; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
const char* cudaGetErrorString(cudaError_t) { return ""; }
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t*, const void*, void**) { return cudaSuccess; }
cudaError_t cudaMalloc(void** p, size_t) { return *p = nullptr, cudaErrorMemoryAllocation; }
cudaError_t cudaFree(void*) { return cudaSuccess; }
cudaError_t cudaMemcpyAsync(void*, const void*, size_t, cudaMemcpyKind, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaMemsetAsync(void*, int, size_t, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaStreamCreateWithFlags(cudaStream_t*, unsigned) { return cudaSuccess; }
cudaError_t cudaStreamDestroy(cudaStream_t) { return cudaSuccess; }
cudaError_t cudaStreamIsCapturing(cudaStream_t, cudaStreamCaptureStatus* s) { return *s = cudaStreamCaptureStatusNone, cudaSuccess; }
cudaError_t cudaStreamSynchronize(cudaStream_t) { return cudaSuccess; }
// what the objects register at their start
void** __cudaRegisterFatBinary(void*) { return nullptr; }
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterFunction(void**, const char*, char*, const char*, int, uint3*, uint3*, dim3*, dim3*, int*) {}
unsigned __cudaPopCallConfiguration(dim3*, dim3*, size_t*, void*) { return 0; }
cudaError_t __cudaGetKernel(void** k, const void*) { return *k = nullptr, cudaSuccess; }
cudaError_t __cudaLaunchKernel(void*, dim3, dim3, void**, size_t, cudaStream_t) { return cudaSuccess; }
}

static size_t parts(size_t rows, size_t cols) {
  size_t bytes = 0;
  if (xp_layernorm_workspace(rows, cols, &bytes) != XP_OK) return 0;
  return bytes / (2 * cols * sizeof(float));
}

int main(int argc, char** argv) {
  if (argc > 1 && !strcmp(argv[1], "devices")) {
    for (int d : {0, 1, 2, 1, 0}) {
      current = d;
      printf("%zu %zu\n", parts(1000000, 1024), parts(1000000, 12000));   // CTAs; clusters of two
    }
    return 0;
  }
  changing = true;
  for (size_t cols : {1024, 12000}) {
    std::vector<size_t> got(16);
    std::vector<std::thread> all;
    std::atomic<bool> go{false};
    for (size_t& g : got)
      all.emplace_back([&g, &go, cols] {
        while (!go.load()) std::this_thread::yield();
        g = parts(1000000, cols);
      });
    go = true;
    for (std::thread& t : all) t.join();
    got.push_back(parts(1000000, cols));
    for (size_t g : got) printf("%zu ", g);
    printf("\n");
  }
  return 0;
}
