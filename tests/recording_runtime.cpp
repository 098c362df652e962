// A stand-in for the HIP runtime that records kernel launches instead of making them, so that
// which kernels a call launches, with which grids and on which device, can be tested without
// a GPU.  It refuses what a device refuses: 2^32 threads or more along x, and more than 64 KiB
// of dynamic LDS for a kernel that was not allowed it on the current device.
#include <cstddef>
#include <cstdint>
#include <map>
#include <set>
#include <string>
#include <utility>
#include <vector>

namespace {
struct Dim {
  uint32_t x, y, z;
};
struct Launch {
  std::string name;
  Dim grid, block;
  size_t lds;
  int device;
};
std::map<const void*, std::string> names;
std::set<std::pair<const void*, int>> allowed;
std::vector<Launch> launches;
int device = 0, refuse_attribute = 0, attributes = 0, last_error = 0;
Dim grid, block;
size_t lds;
void* stream;
constexpr int kInvalidConfiguration = 9, kInvalidValue = 1;
}  // namespace

extern "C" {
void** __hipRegisterFatBinary(const void*) {
  static void* module;
  return &module;
}
void __hipUnregisterFatBinary(void**) {}
void __hipRegisterVar(void**, void*, char*, char*, int, size_t, int, int) {}
void __hipRegisterFunction(void**, const void* host, char*, const char* name, unsigned, void*, void*, void*, void*, int*) {
  names[host] = name;
}
int __hipPushCallConfiguration(Dim g, Dim b, size_t bytes, void* s) {
  grid = g, block = b, lds = bytes, stream = s;
  return 0;
}
int __hipPopCallConfiguration(Dim* g, Dim* b, size_t* bytes, void** s) {
  *g = grid, *b = block, *bytes = lds, *s = stream;
  return 0;
}
int hipLaunchKernel(const void* host, Dim g, Dim b, void**, size_t bytes, void*) {
  const bool threads_ok = uint64_t(g.x) * b.x < uint64_t(1) << 32 && g.x && g.y && g.y < 65536;
  const bool lds_ok = bytes <= (64 << 10) || allowed.count({host, device});
  launches.push_back({names[host], g, b, bytes, device});
  const int e = !threads_ok ? kInvalidConfiguration : !lds_ok ? kInvalidValue : 0;
  if (e) last_error = e;   // an error stays until it is asked for
  return e;
}
int hipFuncSetAttribute(const void* host, int, int) {
  ++attributes;
  if (refuse_attribute) {
    --refuse_attribute;
    return last_error = kInvalidValue;
  }
  allowed.insert({host, device});
  return 0;
}
int hipGetDevice(int* d) {
  *d = device;
  return 0;
}
int hipGetLastError() {
  const int e = last_error;
  last_error = 0;
  return e;
}
const char* hipGetErrorString(int e) { return e == kInvalidConfiguration ? "invalid configuration" : "invalid value"; }

void recorder_device(int d) { device = d; }
void recorder_refuse_attributes(int n) { refuse_attribute = n; }
int recorder_attributes() { return attributes; }
void recorder_clear() { launches.clear(); }
int recorder_launches() { return int(launches.size()); }
const char* recorder_name(int i) { return launches[i].name.c_str(); }
uint32_t recorder_blocks(int i) { return launches[i].grid.x; }
int recorder_launch_device(int i) { return launches[i].device; }
}
