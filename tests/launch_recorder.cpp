// Which kernels a call launches, without a GPU: the library's host code is
// linked with this file, which stands in for the HIP runtime and writes down the
// kernels instead of launching them (tests/test_kernel_choice.py).
//
// One call a line on stdin, its kernels on a line of stdout, tab-separated,
// each with its workgroups:
//   gemm gather grouped M E N K swiglu     (a gather has k == 1)
//   dx grouped M E N K z
//   dw gather grouped M E N K fp32 workspace
//   lora T adapters rank slices N K swiglu
//   combine T k N
//   all                                    (every kernel that there is)
#include <hip/hip_runtime.h>

#include <cxxabi.h>
#include <cstdio>
#include <cstdlib>
#include <iostream>
#include <map>
#include <sstream>
#include <string>
#include <vector>

#include "moesq.h"

static std::map<const void *, std::string> &names() {
  static std::map<const void *, std::string> all;
  return all;
}
static std::vector<std::string> launched;
static dim3 grid_of_call, block_of_call;

static std::string plain(const char *mangled) {
  int status = 0;
  char *s = abi::__cxa_demangle(mangled, nullptr, nullptr, &status);
  std::string name = status ? mangled : s;
  free(s);
  name = name.substr(0, name.find('('));          // without the arguments,
  const size_t at = name.find("moesq::");          // the result's type and the namespace
  return at == std::string::npos ? name : name.substr(at + 7);
}

extern "C" {
void **__hipRegisterFatBinary(const void *) {
  static void *none;
  return &none;
}
void __hipUnregisterFatBinary(void **) {}
void __hipRegisterFunction(void **, const void *host, char *, const char *device, unsigned, void *, void *, dim3 *, dim3 *,
                           int *) {
  names()[host] = plain(device);
}
void __hipRegisterVar(void **, void *, char *, char *, int, size_t, int, int) {}
hipError_t __hipPushCallConfiguration(dim3 grid, dim3 block, size_t, hipStream_t) {
  grid_of_call = grid, block_of_call = block;
  return hipSuccess;
}
hipError_t __hipPopCallConfiguration(dim3 *grid, dim3 *block, size_t *lds, hipStream_t *stream) {
  *grid = grid_of_call, *block = block_of_call, *lds = 0, *stream = nullptr;
  return hipSuccess;
}
hipError_t hipLaunchKernel(const void *f, dim3 grid, dim3, void **, size_t, hipStream_t) {
  launched.push_back(names()[f] + " " + std::to_string(grid.x));
  return hipSuccess;
}
hipError_t hipGetLastError() { return hipSuccess; }
const char *hipGetErrorString(hipError_t) { return ""; }
hipError_t hipGetDevice(int *device) { return *device = 0, hipSuccess; }
hipError_t hipDeviceGetAttribute(int *value, hipDeviceAttribute_t, int) { return *value = 256, hipSuccess; }   // CUs
}

int main() {
  // (buffers far from one another: a call may refuse those that overlap)
  auto at = [](uintptr_t n) { return n << 42; };
  uint16_t *const p[6] = {(uint16_t *)at(1), (uint16_t *)at(2), (uint16_t *)at(3),
                          (uint16_t *)at(4), (uint16_t *)at(5), (uint16_t *)at(6)};
  int32_t *const ip = (int32_t *)at(7);
  float *const fp = (float *)at(8);
  std::string line;
  while (std::getline(std::cin, line)) {
    std::istringstream in(line);
    std::string what;
    in >> what;
    int v[8] = {0};
    for (int &n : v) in >> n;
    launched.clear();
    moesq_status_t st = MOESQ_OK;
    if (what == "gemm") {
      st = moesq_gemm(p[0], v[0] ? ip : nullptr, v[0] ? v[2] : 0, 1, v[1] ? ip : nullptr, v[2], p[1], v[3], v[4], v[5],
                      v[6] ? MOESQ_EPI_SWIGLU : MOESQ_EPI_NONE, p[2], nullptr, nullptr);
    } else if (what == "dx") {
      st = moesq_gemm_dx(p[0], v[0] ? ip : nullptr, v[1], p[1], v[2], v[3], v[4], v[5] ? p[2] : nullptr, p[3], nullptr);
    } else if (what == "dw") {
      const size_t ws = v[7] ? moesq_gemm_dw_workspace_bytes(v[2], v[3], v[4], v[5]) : 0;
      st = moesq_gemm_dw(p[0], p[1], v[0] ? ip : nullptr, v[0] ? v[2] : 0, 1, v[1] ? ip : nullptr, v[2], v[3], v[4], v[5],
                         v[6] ? MOESQ_F32 : MOESQ_BF16, 0, fp, ws ? p[2] : nullptr, ws, nullptr);
    } else if (what == "lora") {
      const moesq_lora_t l = {p[0], p[1], fp, v[1], v[2], v[3], v[4], v[5]};
      st = moesq_lora(p[2], ip, v[0], &l, p[3], v[6] ? MOESQ_EPI_SWIGLU : MOESQ_EPI_NONE, p[4], p[5],
                      moesq_lora_workspace_bytes(v[0], &l), nullptr);
    } else if (what == "combine") {
      st = moesq_unpermute_backward(p[0], p[1], ip, fp, v[0], v[1], v[2], p[2], (float *)p[3], nullptr);
    } else if (what == "all") {
      for (const auto &n : names()) launched.push_back(n.second + " 0");
    } else {
      st = MOESQ_ERR_ARG;
    }
    if (st != MOESQ_OK) {
      printf("error: %s: %s\n", line.c_str(), moesq_last_error());
      return 1;
    }
    for (size_t i = 0; i < launched.size(); ++i) printf("%s%s", i ? "\t" : "", launched[i].c_str());
    printf("\n");
  }
  return 0;
}
