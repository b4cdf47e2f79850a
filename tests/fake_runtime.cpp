// A CUDA runtime of several devices that runs nothing, for the host side of
// the training operators: linked with their objects in place of the runtime.
//
//   fake_runtime devices   parts of a backward pass on devices of 152, 76 and 10 SMs, in turn
//   fake_runtime threads   the same size asked for by 16 threads at once, while the runtime's
//                          answer changes from call to call
//   fake_runtime launches  the largest of what layer norm launches ask for over a sweep of sizes
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
struct {
  size_t launches = 0, smem = 0, threads = 0, cluster = 0, broken = 0;
} seen;
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
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void*, void**) {
  size_t cluster = 1;
  for (unsigned i = 0; i < c->numAttrs; ++i)
    if (c->attrs[i].id == cudaLaunchAttributeClusterDimension) cluster = c->attrs[i].val.clusterDim.x;
  const size_t threads = (size_t)c->blockDim.x * c->blockDim.y * c->blockDim.z;
  ++seen.launches;
  if (c->dynamicSmemBytes > seen.smem) seen.smem = c->dynamicSmemBytes;
  if (threads > seen.threads) seen.threads = threads;
  if (cluster > seen.cluster) seen.cluster = cluster;
  seen.broken += c->gridDim.x == 0 || threads % 32 != 0 || c->gridDim.x % cluster != 0;
  return cudaSuccess;
}
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
  if (argc > 1 && !strcmp(argv[1], "launches")) {
    char* const at = reinterpret_cast<char*>((size_t)1 << 40);   // nothing reads it
    const size_t apart = (size_t)1 << 44;
    for (size_t cols = 1; cols <= XP_LAYERNORM_MAX_COLS; cols += 1 + cols / 37)
      for (size_t width : {cols, (cols + 7) / 8 * 8})
        for (size_t rows = 1; rows <= ((size_t)1 << 20); rows += 1 + rows / 3)
          for (xp_dtype type : {XP_F32, XP_BF16})
            for (size_t off : {0, 4}) {
              if (width > XP_LAYERNORM_MAX_COLS) continue;
              float* const v = reinterpret_cast<float*>(at + 4 * apart);
              const size_t room = (size_t)1 << 40;
              if (xp_layernorm_forward(at + off, width, v, v, at + apart, width, v, v, rows, width, 1e-5f, type, XP_F32, nullptr) != XP_OK ||
                  xp_layernorm_backward(at + off, width, at + 2 * apart, width, v, v, v, at + apart, width, v, v, rows, width, type, XP_F32, 0,
                                        at + 5 * apart, room, nullptr) != XP_OK)
                ++seen.broken;
            }
    printf("%zu %zu %zu %zu %zu\n", seen.launches, seen.smem, seen.threads, seen.cluster, seen.broken);
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
