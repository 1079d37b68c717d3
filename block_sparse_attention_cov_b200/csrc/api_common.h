// api_common.h -- argument checks shared by the C ABI's files (api.cu defines them).
#pragma once

#include <cstdint>

#include "../../include/solattn.h"
#include "kernels.h"

namespace solattn {

constexpr int kMaxDevices = 64;

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

int check_shape(int B, int H, int N, int d);
int check_qkv(const void* q, const void* k, const void* v);
int check_pooled(const solattn_pooled_t* p);
int current_device_sms(int* sms);
int resolve_strides(const solattn_strides_t* in, int B, int H, int N, int d, Strides* out);

}  // namespace solattn
