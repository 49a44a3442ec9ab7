// Drives the C ABI of the attention over a paged cache (gdn_attn_api.cpp) with
// stand-ins for the launchers, under AddressSanitizer and
// UndefinedBehaviorSanitizer: calls that pass validation, and seeded
// descriptors of every kind of size, stride, type and address.  The launchers
// check what reaches them against the sizes they were built for.
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <cstring>

#include "gdn.h"
#include "gdn_api_common.h"
#include "gdn_attn.h"

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

// The multiplication that stands for a division, at the ends and between.
static void check_divide(const Divide& d) {
  for (int64_t n : {(int64_t)0, (int64_t)1, (int64_t)d.d - 1, (int64_t)d.d, (int64_t)d.d + 1, (int64_t)123456789, kMost}) {
    if (n > INT32_MAX) continue;
    const uint32_t hi = (uint32_t)(((uint64_t)d.mul * (uint32_t)n) >> 32);
    CHECK((uint64_t)hi + (uint32_t)n <= UINT32_MAX && (hi + (uint32_t)n) >> d.shift == (uint32_t)n / d.d);
  }
}

hipError_t launch_cache_plan(const PlanParams& p, hipStream_t) {
  ++launches;
  CHECK(p.n >= 0 && p.n <= 1 << 20 && p.t >= 0 && p.t <= kMost && p.width >= 0 && p.free_max >= 0);
  CHECK((__int128)p.width * p.page.d <= kMost && (p.cu || p.t == p.n));
  check_divide(p.page);
  return hipSuccess;
}
hipError_t launch_cache_release(const ReleaseParams& p, hipStream_t) {
  ++launches;
  CHECK(p.n >= 1 && p.n <= 1 << 20 && p.width >= 0 && p.free_max >= 0 && (__int128)p.width * p.page.d <= kMost);
  check_divide(p.page);
  return hipSuccess;
}
hipError_t launch_cache_store(const StoreParams& p, hipStream_t) {
  ++launches;
  CHECK(p.t >= 1 && p.t <= kMost && p.kv >= 1 && p.kv <= 65535 && p.n_slots >= 1 && p.row_shift >= 3 && p.row_shift <= 6);
  CHECK(((uintptr_t)p.k | (uintptr_t)p.v | (uintptr_t)p.k_cache | (uintptr_t)p.v_cache) % 16 == 0);
  CHECK((p.t == 1 || p.k_st % 16 == 0) && (p.kv == 1 || p.vc_sh % 16 == 0));
  return hipSuccess;
}
int attn_tile_rows(bool bf16, int) { return bf16 ? 128 : 64; }
static void check_attn(int d, const AttnParams& p) {
  ++launches;
  CHECK((d == 64 || d == 128 || d == 256) && p.heads >= 1 && p.heads <= 65535 && p.kv >= 1 && p.heads == p.kv * p.group);
  CHECK(((uintptr_t)p.q | (uintptr_t)p.k | (uintptr_t)p.v | (uintptr_t)p.out) % 16 == 0 || (p.table && p.pages == 0));
  CHECK(p.window >= 0 && p.sinks >= 0 && p.scale == p.scale && p.scale - p.scale == 0.f);
  CHECK(!p.table == !p.lens);
  if (p.table) {
    CHECK((int64_t)p.width * p.page.d == p.max_len && p.max_len <= kMost && p.pages >= 0);
    check_divide(p.page);
  }
}
hipError_t launch_attn_prefill(bool bf16, int d, const AttnParams& p, hipStream_t) {
  check_attn(d, p);
  const int rows = bf16 ? 128 : 64;
  CHECK(p.t_total >= 1 && p.n_seq >= 1 && (p.cu || (int64_t)p.n_seq * p.seq_len == p.t_total));
  const int64_t tiles = p.cu ? (int64_t)p.t_total / rows + p.n_seq : (int64_t)p.n_seq * ((p.seq_len + rows - 1) / rows);
  CHECK(tiles >= 1 && tiles * p.heads * 512 < (int64_t)1 << 32);
  return hipSuccess;
}
int attn_decode_waves(bool, int d) { return 256 * (d == 64 ? 8 : d == 128 ? 4 : 2); }
hipError_t launch_attn_decode(bool, int d, const AttnParams& p, hipStream_t) {
  check_attn(d, p);
  CHECK(p.table && p.n_seq >= 1 && p.n_seq <= 1 << 20 && p.waves >= 1 && (p.waves & (p.waves - 1)) == 0);
  CHECK((char*)p.chains - (char*)p.parts >= (int64_t)2 * p.waves * attn_part_floats(d) * 4);
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
  t.dtype = rnd() % 60 ? dtype : (int32_t)pick({0, 1, 2, 3, 4, 5, 6, -1, INT32_MAX});
  t.ndim = (int)shape.size();
  const bool odd = rnd() % 5 == 0;
  for (int i = 0; i < t.ndim; ++i) t.shape[i] = odd ? size_near(shape.begin()[i]) : shape.begin()[i];
  __int128 acc = 1;
  for (int i = t.ndim - 1; i >= 0; --i) {
    t.stride[i] = acc > INT64_MAX ? INT64_MAX : (int64_t)acc;
    if (t.shape[i] > 0) acc *= t.shape[i];
    if (acc > INT64_MAX) acc = INT64_MAX;
  }
  if (rnd() % 10 == 0) t.stride[rnd() % t.ndim] = pick({0, -1, 1, 3, 8, 64, 1 << 24, (1 << 24) + 8, (int64_t)1 << 40, INT64_MAX, INT64_MIN});
  if (rnd() % 60 == 0) t.ndim = (int)pick({0, 1, 2, 3, 4, 5, -1});
  address += (uintptr_t)1 << 36;
  t.data = (void*)(rnd() % 30 ? address : (uintptr_t)pick({0, (int64_t)address + 1, (int64_t)address + 8, 0x100000000}));
  return t;
}

static bool known(int rc) { return rc <= 0 && rc >= -8; }

int main() {
  long passed = 0, calls = 0;
  for (int i = 0; i < 400000; ++i) {
    const int32_t type = rnd() % 2 ? GDN_DTYPE_BF16 : GDN_DTYPE_F32;
    const int64_t N = pick({0, 1, 3, 300, 1 << 20, (1 << 20) + 1}), M = pick({0, 1, 8, 1000, 1 << 20}), F = pick({0, 1, 100, 1 << 20});
    const int64_t T = pick({0, 1, 5, 1000, 1 << 20, gdn::kMost, gdn::kMost + 1});
    const int64_t page = pick({1, 16, 16, 48, 64, 1 << 10, 1 << 20}), pages = pick({0, 1, 7, 1 << 16}), kv = pick({1, 2, 8, 4095}), H = kv * pick({1, 2, 7, 16, 17});
    const int64_t d = pick({64, 128, 256, 96});
    const int32_t psz = (int32_t)(rnd() % 12 ? page : pick({0, -1, INT32_MAX, INT32_MIN, 1 << 30}));
    gdn_tensor table = tensor(GDN_DTYPE_I32, {N, M}), lens = tensor(GDN_DTYPE_I32, {N}), free = tensor(GDN_DTYPE_I32, {F}), left = tensor(GDN_DTYPE_I32, {1});
    gdn_tensor kc = tensor(type, {pages, page, kv, d}), vc = tensor(type, {pages, page, kv, d});
    gdn_attn_options o;
    gdn_attn_default_options(&o);
    if (rnd() % 4 == 0) {
      const float scales[] = {0.f, 1.f, -1.f, 1e-38f, 1e19f, 1e20f, -1e30f, __builtin_inff(), __builtin_nanf("")};
      o.scale = scales[rnd() % 9];
      o.window = (int32_t)pick({0, 1, 1000, INT32_MAX, -1});
      o.sinks = (int32_t)pick({0, 1, 1000, INT32_MAX, -1});
    }
    int rc;
    ++calls;
    switch (rnd() % 5) {
      case 0: {
        const bool one = rnd() % 2;
        gdn_tensor ctx = tensor(GDN_DTYPE_I32, {N}), cu = tensor(rnd() % 2 ? GDN_DTYPE_I32 : GDN_DTYPE_I64, {N + 1}), slots = tensor(GDN_DTYPE_I64, {one ? N : T}),
                   out = tensor(GDN_DTYPE_I32, {1});
        rc = gdn_cache_plan(&ctx, one ? nullptr : &cu, &table, &free, &left, psz, rnd() % 2 ? &lens : &ctx, &slots, rnd() % 2 ? &out : &left, nullptr);
        break;
      }
      case 1: {
        gdn_tensor done = tensor(GDN_DTYPE_I32, {N});
        rc = gdn_cache_release(&done, &lens, &table, &free, &left, psz, nullptr);
        break;
      }
      case 2: {
        gdn_tensor k = tensor(type, {T, kv, d}), v = tensor(type, {T, kv, d}), slots = tensor(GDN_DTYPE_I64, {T});
        if (rnd() % 4 == 0) {  // the halves of one allocation
          vc = kc;
          vc.data = (char*)kc.data + pick({0, 16, 2 * d, 4 * d, 2 * d * kv, 2 * d * kv * page});
        }
        rc = gdn_cache_store(&k, &v, &slots, &kc, &vc, nullptr);
        break;
      }
      case 3: {
        const bool batched = rnd() % 3 == 0, cached = rnd() % 2;
        const int64_t B = batched ? pick({1, 2, 300}) : 1;
        gdn_tensor cu = tensor(rnd() % 2 ? GDN_DTYPE_I32 : GDN_DTYPE_I64, {N + 1});
        gdn_tensor q = batched ? tensor(type, {B, T, H, d}) : tensor(type, {T, H, d}), out = batched ? tensor(type, {B, T, H, d}) : tensor(type, {T, H, d});
        gdn_tensor k = batched ? tensor(type, {B, T, kv, d}) : tensor(type, {T, kv, d}), v = batched ? tensor(type, {B, T, kv, d}) : tensor(type, {T, kv, d});
        rc = gdn_attn_prefill(&q, cached ? &kc : &k, cached ? &vc : &v, rnd() % 3 ? &cu : nullptr, cached ? &table : nullptr, cached ? &lens : nullptr, &out,
                              rnd() % 2 ? &o : nullptr, nullptr);
        break;
      }
      default: {
        gdn_tensor q = tensor(type, {N, H, d}), out = tensor(type, {N, H, d});
        size_t need = 0;
        const int sized = gdn_attn_workspace_size(&q, &need);
        CHECK(known(sized));
        rc = gdn_attn_decode(&q, &kc, &vc, &table, &lens, &out, rnd() % 2 ? &o : nullptr,
                             (void*)(uintptr_t)pick({0x40000000, 0x40000000, 0x40000000, 0, 0x40000010}), rnd() % 8 ? need : need / 2, nullptr);
        CHECK(sized == GDN_OK || rc != GDN_OK);
      }
    }
    CHECK(known(rc));
    passed += rc == GDN_OK;
  }
  printf("%ld calls, %ld valid, %d launches, %d failure(s)\n", calls, passed, launches, failures);
  return failures || passed < 10000 ? 1 : 0;
}
