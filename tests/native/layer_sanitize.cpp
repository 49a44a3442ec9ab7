// Drives the C ABI of the operators around the projections
// (gdn_layer_api.cpp) with stand-ins for the launchers, under AddressSanitizer
// and UndefinedBehaviorSanitizer: calls that pass validation, and seeded
// descriptors of every kind of size, stride, type and address.  The launchers
// check what reaches them against the sizes they were built for.
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <vector>

#include "gdn.h"
#include "gdn_api_common.h"
#include "gdn_layer.h"

static int failures = 0, launches = 0;
#define CHECK(c) \
  do { \
    if (!(c)) { ++failures; printf("line %d: %s\n", __LINE__, #c); } \
  } while (0)

namespace gdn {

int api_fail(int status, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  return status;
}
void api_clear_error() {}
int api_debug_check_cu(const gdn_tensor*, int64_t, int64_t, hipStream_t) { return GDN_OK; }

constexpr int64_t kMost = ((int64_t)1 << 31) - ((int64_t)1 << 21);
hipError_t launch_short_conv(bool, bool vec, const ShortConvParams& p, hipStream_t) {
  ++launches;
  CHECK(p.width >= 1 && p.width <= 4 && p.d >= 1 && p.n_seq >= 1 && p.t_total >= 0 && p.t_total <= kMost);
  CHECK(p.cu || (int64_t)p.n_seq * p.seq_len == p.t_total);
  CHECK(!vec || (uintptr_t)p.x % 16 == 0);
  return hipSuccess;
}
hipError_t launch_add_rms_norm(bool, bool, const NormParams& p, hipStream_t) {
  ++launches;
  CHECK(p.rows >= 1 && p.d >= 1 && p.d <= 65536 && !p.out_q == !p.scales);
  return hipSuccess;
}
int ssm_target_groups() { return 512; }
int ssm_group_heads(bool bf16, int p, int group) { return bf16 && p == 64 && group % 2 == 0 ? 2 : 1; }
hipError_t launch_ssm_table(const SsmTable& p, hipStream_t) {
  ++launches;
  CHECK(p.seg_len >= 64 && p.seg_len % 64 == 0 && p.max_segs >= p.n_seq && !p.cuts == !p.cut_table);
  return hipSuccess;
}
hipError_t launch_ssm_states(bool, int, int, const SsmParams& p, hipStream_t) {
  ++launches;
  CHECK(p.slots && p.seg_decay && p.max_cuts >= 1 && p.max_cut_segs >= 2 && p.max_cut_segs <= p.max_segs);
  return hipSuccess;
}
hipError_t launch_ssm_scan(bool, int n, int pp, const SsmParams& p, hipStream_t) {
  ++launches;
  CHECK(n >= 16 && n <= 128 && pp >= 16 && pp <= 128 && p.heads >= 1 && p.heads % p.group == 0 && p.max_segs >= 1);
  CHECK(p.packed ? p.table && p.seg_off : p.n_seq * (int64_t)p.segs_per_seq == p.max_segs);
  CHECK(p.x_st >= 0 && p.x_st <= 1 << 24 && p.o_st <= 1 << 24);
  return hipSuccess;
}
hipError_t launch_ssm_step(bool, int, int, const SsmStepParams& p, hipStream_t) {
  ++launches;
  CHECK(p.n >= 1 && p.heads >= 1 && p.heads % p.group == 0);
  return hipSuccess;
}

}  // namespace gdn

extern "C" const char* hipGetErrorString(hipError_t) { return "host-only build"; }

static uint64_t state = 1;
static uint64_t rnd() {
  state = state * 6364136223846793005ull + 1442695040888963407ull;
  return state >> 33;
}
static int64_t pick(std::initializer_list<int64_t> v) { return v.begin()[rnd() % v.size()]; }

// Mostly the wanted size, now and then another one.
static int64_t size_near(int64_t want) {
  switch (rnd() % 24) {
    case 0: return 0;
    case 1: return 1;
    case 2: return want + 1;
    case 3: return pick({-1, (int64_t)1 << 31, ((int64_t)1 << 31) - 1, (int64_t)1 << 40, INT64_MAX, INT64_MIN, 65536});
  }
  return want;
}

static uintptr_t address = 0x100000000;
static gdn_tensor tensor(int32_t dtype, std::initializer_list<int64_t> shape) {
  gdn_tensor t;
  memset(&t, 0, sizeof t);
  t.dtype = rnd() % 40 ? dtype : (int32_t)pick({0, 1, 2, 3, 4, 5, 6, -1, INT32_MAX});
  t.ndim = (int)shape.size();
  const bool odd = rnd() % 3 == 0;
  for (int i = 0; i < t.ndim; ++i) t.shape[i] = odd ? size_near(shape.begin()[i]) : shape.begin()[i];
  __int128 acc = 1;
  for (int i = t.ndim - 1; i >= 0; --i) {
    t.stride[i] = acc > INT64_MAX ? INT64_MAX : (int64_t)acc;
    if (t.shape[i] > 0) acc *= t.shape[i];
    if (acc > INT64_MAX) acc = INT64_MAX;
  }
  if (rnd() % 6 == 0) t.stride[rnd() % t.ndim] = pick({0, -1, 1, 3, 8, 64, 1 << 24, (1 << 24) + 8, (int64_t)1 << 40, INT64_MAX, INT64_MIN});
  if (rnd() % 40 == 0) t.ndim = (int)pick({0, 1, 2, 3, 4, 5, -1});
  address += (uintptr_t)1 << 36;
  t.data = (void*)(rnd() % 20 ? address : (uintptr_t)pick({0, (int64_t)address + 1, (int64_t)address + 8, 0x100000000}));
  return t;
}

static bool known(int rc) { return rc <= 0 && rc >= -8; }

int main() {
  long passed = 0, calls = 0;
  for (int i = 0; i < 400000; ++i) {
    const int32_t type = rnd() % 2 ? GDN_DTYPE_BF16 : GDN_DTYPE_F32;
    const int64_t T = pick({0, 1, 5, 64, 65, 1000, 1 << 20, gdn::kMost, gdn::kMost + 1}), B = pick({1, 1, 2, 3, 1000});
    const bool batched = rnd() % 3 == 0;
    gdn_tensor cu = tensor(rnd() % 2 ? GDN_DTYPE_I32 : GDN_DTYPE_I64, {pick({2, 2, 3, 300, 1 << 20, gdn::kMost + 1})});
    const gdn_tensor* pcu = rnd() % 2 ? &cu : nullptr;
    const int64_t seqs = pcu && cu.shape[0] > 1 ? cu.shape[0] - 1 : batched ? B : 1;
    int rc;
    ++calls;
    switch (rnd() % 4) {
      case 0: {
        const int64_t D = pick({1, 8, 1001, 6144, gdn::kMost, gdn::kMost + 1}), W = pick({1, 2, 3, 4, 4, 5});
        gdn_tensor x = batched ? tensor(type, {B, T, D}) : tensor(type, {T, D});
        gdn_tensor out = batched ? tensor(type, {B, T, D}) : tensor(type, {T, D});
        gdn_tensor w = tensor(GDN_DTYPE_F32, {D, W}), si = tensor(type, {seqs, W - 1, D}), so = tensor(type, {seqs, W - 1, D});
        rc = gdn_short_conv(&x, &w, rnd() % 2 ? (const float*)0x10000 : nullptr, pcu, rnd() % 2 ? &si : nullptr,
                            rnd() % 3 ? rnd() % 2 ? &so : &si : nullptr, &out, rnd() % 20 ? rnd() % 2 : 2u, nullptr);
        break;
      }
      case 1: {
        const int64_t G = pick({1, 2, 3, 16}), H = G * pick({1, 2, 3, 4096}), N = pick({16, 32, 64, 128, 48}), P = pick({16, 32, 64, 128, 256});
        gdn_tensor x = batched ? tensor(type, {B, T, H, P}) : tensor(type, {T, H, P});
        gdn_tensor out = batched ? tensor(type, {B, T, H, P}) : tensor(type, {T, H, P});
        gdn_tensor b = batched ? tensor(type, {B, T, G, N}) : tensor(type, {T, G, N});
        gdn_tensor c = batched ? tensor(type, {B, T, G, N}) : tensor(type, {T, G, N});
        gdn_tensor dt = batched ? tensor(GDN_DTYPE_F32, {B, T, H}) : tensor(GDN_DTYPE_F32, {T, H});
        gdn_tensor init = tensor(GDN_DTYPE_F32, {seqs, H, N, P}), fin = tensor(GDN_DTYPE_F32, {seqs, H, N, P});
        gdn_ssm_options o;
        gdn_ssm_default_options(&o);
        o.segment_blocks = (int32_t)pick({0, 0, -1, 1, 2, 100, INT32_MAX, -2, INT32_MIN});
        if (rnd() % 2) o.a_log = (const float*)0x20000;
        size_t need = 0;
        const int sized = gdn_ssm_workspace_size(&x, &b, pcu, &o, &need);
        CHECK(known(sized));
        rc = gdn_ssm_prefill(&x, &dt, &b, &c, pcu, rnd() % 2 ? &init : nullptr, &out, rnd() % 3 ? rnd() % 2 ? &fin : &init : nullptr,
                             &o, (void*)(uintptr_t)pick({0x40000000, 0x40000000, 0, 0x40000010}), rnd() % 8 ? need : need / 2, nullptr);
        CHECK(sized == GDN_OK || rc != GDN_OK);
        break;
      }
      case 2: {
        const int64_t n = pick({0, 1, 3, 256, 1 << 20, gdn::kMost, gdn::kMost + 1});
        const int64_t G = pick({1, 2, 16}), H = G * pick({1, 3, 4095}), N = pick({16, 128, 8}), P = pick({16, 128, 8});
        gdn_tensor x = tensor(type, {n, H, P}), out = tensor(type, {n, H, P}), dt = tensor(GDN_DTYPE_F32, {n, H});
        gdn_tensor b = tensor(type, {n, G, N}), c = tensor(type, {n, G, N}), st = tensor(GDN_DTYPE_F32, {n, H, N, P});
        rc = gdn_ssm_decode(&x, &dt, &b, &c, &st, &out, nullptr, nullptr);
        break;
      }
      default: {
        const int64_t R = pick({0, 1, 5, 1000, ((int64_t)1 << 31) - 1}), D = pick({1, 8, 100, 128, 6144, 65536, 65537});
        gdn_tensor x = tensor(type, {R, D}), r = tensor(type, {R, D}), ro = tensor(type, {R, D}), out = tensor(type, {R, D});
        gdn_tensor q = tensor(GDN_E4M3, {R, D}), s = rnd() % 2 ? tensor(GDN_DTYPE_F32, {R}) : tensor(GDN_DTYPE_F32, {R, (D + 127) / 128});
        const bool eight = rnd() % 2;
        rc = gdn_add_rms_norm(&x, rnd() % 2 ? &r : nullptr, rnd() % 2 ? (const float*)0x30000 : nullptr, 1e-6f, rnd() % 3 ? rnd() % 2 ? &ro : &x : nullptr,
                              rnd() % 2 ? &out : nullptr, eight ? &q : nullptr, eight || rnd() % 30 == 0 ? &s : nullptr, nullptr);
      }
    }
    CHECK(known(rc));
    passed += rc == GDN_OK;
  }
  printf("%ld calls, %ld valid, %d launches, %d failure(s)\n", calls, passed, launches, failures);
  return failures || passed < 10000 ? 1 : 0;
}
