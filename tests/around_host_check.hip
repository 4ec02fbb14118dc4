// Host-only check of what the calls around the products hand to their kernels
// (built and run by tests/test_around_host.py; no GPU code is executed).
//
// The library's own host code is compiled here with the HIP runtime's queries
// and launches replaced by recorders: the C entries are called with made-up
// addresses and what would be launched is compared with what is expected.
// One line is printed for each disagreement, and the exit status says whether
// there was any.
#include <hip/hip_runtime.h>

#include <cstdio>
#include <cstring>
#include <map>
#include <mutex>
#include <utility>
#include <vector>

namespace fake {
int device = 0;
struct Launch {
  const void* kernel;
  dim3 grid, block;
  size_t lds;
};
std::vector<Launch> launches;
template <typename A>
struct Args {
  static A last;  // of the kernels that take an A first
};
template <typename A>
A Args<A>::last{};

hipError_t get_device(int* d) {
  *d = device;
  return hipSuccess;
}
hipError_t get_properties(hipDeviceProp_t* p, int) {
  memset(p, 0, sizeof(*p));
  strcpy(p->gcnArchName, "gfx950");
  return hipSuccess;
}
hipError_t last_error() { return hipSuccess; }
// a kernel's limit of dynamic and static LDS, on each device
std::map<std::pair<int, const void*>, int> lds_limits;
std::mutex lds_mutex;
hipError_t set_attribute(const void* kernel, hipFuncAttribute what, int value) {
  if (what != hipFuncAttributeMaxDynamicSharedMemorySize) return hipErrorInvalidValue;
  std::lock_guard<std::mutex> lk(lds_mutex);
  lds_limits[{device, kernel}] = value;
  return hipSuccess;
}
int lds_limit(const void* kernel) {
  const auto it = lds_limits.find({device, kernel});
  return it == lds_limits.end() ? 64 << 10 : it->second;
}
template <typename A, typename... More>
void launch(const void* kernel, dim3 grid, dim3 block, size_t lds, const A& a, const More&...) {
  launches.push_back(Launch{kernel, grid, block, lds});
  Args<A>::last = a;
}
}  // namespace fake

#undef hipGetDeviceProperties
#define hipGetDeviceProperties fake::get_properties
#define hipFuncSetAttribute fake::set_attribute
#define hipGetDevice fake::get_device
#define hipGetLastError fake::last_error
#undef hipLaunchKernelGGL
#define hipLaunchKernelGGL(kernel, grid, block, lds, stream, ...) \
  fake::launch(reinterpret_cast<const void*>(kernel), grid, block, lds, __VA_ARGS__)

#include "rq_api.hip"
#include "rq_logits.hip"
#include "rq_lora.hip"
#include "rq_mv.hip"
#include "rq_wkv.hip"

namespace {
int bad = 0;
void expect(bool ok, const char* what) {
  if (!ok) printf("WRONG %s\n", what), bad++;
}
char* at(size_t i) { return reinterpret_cast<char*>((size_t)0x7F0000000000 + (i << 32)); }
template <typename T>
T* array_at(size_t i) {
  return reinterpret_cast<T*>(at(i));
}
}  // namespace

// A group whose first pointer is NULL is left out whole: its other pointers
// are not read, whatever they are.
static void logits_groups() {
  rq_logits_args g{};
  g.logits = array_at<const float>(0);
  g.out = array_at<float>(1);
  g.M = 4;
  g.V = 1000;
  g.history_offsets = array_at<const int>(2);
  g.prompt = array_at<const int>(3);
  g.repetition = array_at<const float>(4);
  g.presence = array_at<const float>(5);
  g.frequency = array_at<const float>(6);
  g.bias = array_at<const float>(7);
  g.bias_offsets = array_at<const int>(8);
  g.mask_ids = array_at<const int>(9);
  expect(rq_logits(&g, nullptr, 0, nullptr) == RQ_OK, "groups left out are accepted");
  const rq::LogitsArgs& a = fake::Args<rq::LogitsArgs>::last;
  expect(!a.history && !a.bias_ids && !a.masks, "groups left out");
  expect(!a.history_offsets && !a.prompt, "history's lists without a history");
  expect(!a.repetition && !a.presence && !a.frequency, "penalties without a history");
  expect(!a.bias && !a.bias_offsets && !a.mask_ids, "lists of biases and masks left out");
  g.history = array_at<const int>(10);
  g.history_len = 100;
  expect(rq_logits(&g, nullptr, 0, nullptr) == RQ_OK, "a history is accepted");
  expect(a.history == g.history && a.history_offsets == g.history_offsets &&
             a.prompt == g.prompt && a.repetition == g.repetition && a.presence == g.presence &&
             a.frequency == g.frequency && a.history_len == 100,
         "a history's lists reach the kernel");
}

// A kernel's limit is raised where its dynamic and its static LDS (up to 128
// bytes, one record for each wave) together pass 64 KiB.
static void logits_lds() {
  rq_logits_args g{};
  g.logits = array_at<const float>(0);
  g.out = array_at<float>(16);
  g.history = array_at<const int>(32);
  g.history_offsets = array_at<const int>(33);
  const int sizes[][2] = {{128, 65536}, {256, 32768}, {256, 65536}, {1, 65536}, {64, 65536}};
  for (const auto& mv : sizes) {
    g.M = mv[0];
    g.V = mv[1];
    expect(rq_logits(&g, nullptr, 0, nullptr) == RQ_OK, "history only");
    const fake::Launch& l = fake::launches.back();
    expect((int)l.lds + 128 <= fake::lds_limit(l.kernel), "LDS within its limit");
  }
}

// The limit is a device's: every device a kernel runs on has it raised.
static void lds_on_every_device() {
  rq_logits_args g{};
  g.logits = array_at<const float>(0);
  g.out = array_at<float>(16);
  g.history = array_at<const int>(32);
  g.history_offsets = array_at<const int>(33);
  g.M = 200;
  g.V = 65536;
  rq::Problem p{array_at<const void>(0), array_at<const void>(1), nullptr, array_at<const void>(2),
                array_at<float>(3), 4, 4096, 16384, 64, rq::FMT_S4};
  const rq::Problem* const ps[] = {&p};
  for (fake::device = 0; fake::device < 64; fake::device += 21) {
    expect(rq_logits(&g, nullptr, 0, nullptr) == RQ_OK, "logits on another device");
    const fake::Launch l = fake::launches.back();
    expect((int)l.lds + 128 <= fake::lds_limit(l.kernel), "LDS of rq_logits on another device");
    expect(rq::launch_mv_many(ps, 1, nullptr) == hipSuccess, "products on another device");
    const fake::Launch m = fake::launches.back();
    expect((int)m.lds > 64 << 10 && (int)m.lds <= fake::lds_limit(m.kernel),
           "LDS of the decode kernel on another device");
  }
  fake::device = 0;
}

// Launches of rq_wkv7: token by token, in chunks, or one of each.  Fewer tokens
// than sequences say that some are empty, and then any of the others may be long.
static size_t wkv_launches(int T, int sequences, int H) {
  const size_t before = fake::launches.size();
  expect(rq_wkv7(at(0), at(8), at(16), at(24), at(32), at(40), RQ_TYPE_F32, nullptr,
                 array_at<float>(48), array_at<const int>(56), array_at<const int>(57), T, H,
                 sequences, 0, nullptr) == RQ_OK,
         "wkv7");
  return fake::launches.size() - before;
}
static void wkv_empty_sequences() {
  expect(wkv_launches(48, 64, 4) == 2, "48 tokens in 64 slots");
  expect(wkv_launches(255, 256, 64) == 2, "255 tokens in 256 slots");
  expect(wkv_launches(20, 4096, 1) == 2, "20 tokens in 4096 slots");
  expect(wkv_launches(7, 64, 1) == 1, "7 tokens, none long");
  expect(wkv_launches(15, 64, 4) == 1, "15 tokens of many heads, none long");
  expect(wkv_launches(64, 64, 64) == 1, "a single token in every slot");
  expect(wkv_launches(70, 64, 64) == 1, "few more tokens than sequences");
  expect(wkv_launches(300, 64, 64) == 2, "both kinds");
  expect(wkv_launches(4096, 1, 64) == 1, "one prompt");
}

// Any number of adapters an int32 id can name: a block's groups are no more than
// its rows, and few-row kernels are taken where rows mostly have their own.
static void lora_many_adapters() {
  for (int adapters : {1, 3, 100, 1 << 28, 2147483647}) {
    for (int M : {1, 4, 64, 100}) {
      rq_lora_problem p{at(0), at(8), at(16), nullptr, array_at<float>(24), 4096, 4096};
      size_t need = 0;
      expect(rq_lora_workspace_size(&p, 1, M, adapters, 16, &need) == RQ_OK, "workspace size");
      expect(rq_lora(&p, 1, M, array_at<const int>(32), array_at<const int>(40), nullptr, adapters,
                     48, 16, at(64), need, nullptr) == RQ_OK,
             "lora");
      const size_t n = fake::launches.size();
      const int rows = M < 64 ? M : 64;
      const int most = adapters < rows ? adapters + 1 : rows;
      for (size_t i = n - 2; i < n; i++) {
        const dim3 g = fake::launches[i].grid;
        expect(g.z >= 1 && (int)g.z <= most && g.y == (M + 63u) / 64, "groups of a block of rows");
      }
      if (M == 64 && adapters >= 100) {  // the same kernel from 100 adapters on
        static const void* const first = fake::launches[n - 1].kernel;
        expect(fake::launches[n - 1].kernel == first, "few rows an adapter");
      }
    }
  }
}

int main() {
  lora_many_adapters();
  wkv_empty_sequences();
  logits_groups();
  logits_lds();
  lds_on_every_device();
  printf("wrong=%d\n", bad);
  return bad ? 1 : 0;
}
