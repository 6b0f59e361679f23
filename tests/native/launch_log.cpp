// Stands in for the HIP runtime's launches where there is no device: a library that is loaded after this one
// (with RTLD_GLOBAL) registers its kernels here, and a launch writes down its kernel's name, grid and block instead.
#include <cstdint>
#include <map>
#include <string>

namespace {
std::map<const void*, std::string>& kernels() {
  static std::map<const void*, std::string> k;
  return k;
}
std::string g_log, g_out;
}  // namespace

struct Dim3 {
  uint32_t x, y, z;
};

extern "C" {
void** __hipRegisterFatBinary(const void*) {
  static void* none;
  return &none;
}
void __hipRegisterFunction(void**, const void* host, char*, const char* name, unsigned, void*, void*, void*, void*, int*) { kernels()[host] = name; }
void __hipRegisterVar(void**, void*, char*, char*, int, size_t, int, int) {}
void __hipUnregisterFatBinary(void**) {}
int hipLaunchKernel(const void* f, Dim3 grid, Dim3 block, void**, size_t, void*) {
  const auto it = kernels().find(f);
  const uint64_t threads = (uint64_t)block.x * block.y * block.z * grid.x * grid.y * grid.z;
  g_log += (it == kernels().end() ? "?" : it->second) + " " + std::to_string(grid.x) + " " + std::to_string(grid.y) + " " +
           std::to_string(grid.z) + " " + std::to_string(threads) + "\n";
  return 0;
}
int hipGetLastError() { return 0; }

// The launches since the last call, one a line: name, grid, threads.
const char* launch_log() {
  g_out.swap(g_log);
  g_log.clear();
  return g_out.c_str();
}
// The names of all kernels, one a line.
const char* launch_kernels() {
  g_out.clear();
  for (const auto& k : kernels()) g_out += k.second + "\n";
  return g_out.c_str();
}
}
