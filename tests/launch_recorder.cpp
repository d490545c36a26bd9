// Stand-ins for the HIP runtime calls that a training operator's entry makes,
// preloaded before the library on a machine without a GPU: every launch is noted
// (kernel, grid, block) and nothing runs.  A launch that the runtime would
// refuse, 2^32 threads or more along an axis or a block of more than 1024, is
// refused here too.
#include <cxxabi.h>

#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <map>
#include <string>

struct dim3 {
  uint32_t x, y, z;
};

namespace {
constexpr int kInvalidConfiguration = 9;
std::map<const void*, std::string> g_names;
std::string g_log, g_taken;
int g_error = 0;
dim3 g_grid, g_block;
size_t g_shared;
void* g_stream;

int refuse(int e) {
  if (e) g_error = e;
  return e;
}
}  // namespace

extern "C" {

void** __hipRegisterFatBinary(const void*) {
  static void* module;
  return &module;
}
void __hipUnregisterFatBinary(void**) {}
void __hipRegisterVar(void**, void*, char*, char*, int, size_t, int, int) {}
void __hipRegisterFunction(void**, const void* host, char*, const char* device, unsigned, void*, void*, void*, void*, int*) {
  int status = 0;
  char* text = abi::__cxa_demangle(device, nullptr, nullptr, &status);
  g_names[host] = status == 0 ? text : device;
  std::free(text);
}
int __hipPushCallConfiguration(dim3 grid, dim3 block, size_t shared, void* stream) {
  g_grid = grid;
  g_block = block;
  g_shared = shared;
  g_stream = stream;
  return 0;
}
int __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* shared, void** stream) {
  *grid = g_grid;
  *block = g_block;
  *shared = g_shared;
  *stream = g_stream;
  return 0;
}
int hipLaunchKernel(const void* f, dim3 grid, dim3 block, void**, size_t, void*) {
  char line[160];
  std::snprintf(line, sizeof line, "%u %u %u %u %u %u ", grid.x, grid.y, grid.z, block.x, block.y, block.z);
  g_log += line + g_names[f] + "\n";
  bool ok = uint64_t(block.x) * block.y * block.z <= 1024;
  for (auto [g, b] : {std::pair(grid.x, block.x), std::pair(grid.y, block.y), std::pair(grid.z, block.z)})
    ok = ok && g > 0 && b > 0 && uint64_t(g) * b < (uint64_t(1) << 32);
  return refuse(ok ? 0 : kInvalidConfiguration);
}
int hipGetLastError() {
  const int e = g_error;
  g_error = 0;
  return e;
}
int hipGetDevice(int* dev) {
  *dev = 0;
  return 0;
}
int hipStreamIsCapturing(void*, int* status) {
  *status = 0;
  return 0;
}

// The launches since the last call, one a line.
const char* recorder_take() {
  g_taken.swap(g_log);
  g_log.clear();
  return g_taken.c_str();
}
}
