// Host helpers of the C ABI, shared by its source files (defined in api.cpp).
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace dg {

// Byte offsets a kernel may use inside one buffer range: below the
// out-of-range marker (0xFFFFFF00) the kernels give lanes outside a tile.
constexpr int64_t kOffLim = (int64_t)0xFFFFFF00 - 4096;
constexpr int64_t kMaxGroups = 1024;

// Sets this thread's error text and returns `code`; ok() clears it.
int fail(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
int ok();

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Checks that a HIP device is current and is gfx950; returns its CU count (>0) or fails.
int check_device(int* cus);
// CU count of the current device for the planning queries (256 without a device).
int query_cus();
// The device's CU count under the cap of dg_set_num_cus.
int effective_cus(int device_cus);
// DG_PRINT_CONFIGS is set
bool print_configs();

// Under DG_CHECK_LAYOUT: whether every aligned 128-row block of m_indices holds rows of at most one expert.
int check_contiguous_layout(const int32_t* m_indices, int64_t M_total, int64_t G, void* stream);

// Workspace bytes and plan texts of the operations of api_moe.cpp (0 / "" for others).
size_t moe_workspace_size(int op, int64_t rows, int64_t N, int64_t K, int64_t G, int cus);
int moe_describe_plan(int op, int64_t rows, int64_t N, int64_t K, int64_t G, int cus, char* buf, size_t n);

}  // namespace dg
