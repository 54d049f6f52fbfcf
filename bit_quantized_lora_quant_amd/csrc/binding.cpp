// For the Python binding alone, not part of the C ABI: where many torch tensors lie and
// how, in one call.  torch publishes a table of C functions that look into a tensor
// (DLPack's exchange interface, version 1); asking a tensor for its address, type, shape
// and strides from Python takes four calls of 50 to 100 ns each, longer for 1344 tensors
// than the GPU needs to update them.
#include <cstdint>

namespace {

struct View {                 // DLTensor
  void* data;
  int32_t device_type, device_id;
  int32_t ndim;
  uint8_t code, bits;
  uint16_t lanes;
  int64_t* shape;
  int64_t* strides;
  uint64_t byte_offset;
};
struct Table {                // DLPackExchangeAPI
  uint32_t major, minor;
  void* previous;
  void* allocate;
  void* take;
  void* give;
  int (*view)(void* object, View* out);   // nullable; not 0: a Python exception is set
  void* stream;
};

}  // namespace

// at[i]: tensor i's address; layout[6 i ..]: its type, device, rows, columns (-1 of all but
// a matrix), row and column stride (0 where no two elements are that far apart).  table is torch's; with n == 0 whether it can
// be used.  Called with the interpreter's lock held.  Returns 0 or -1 (exception set).
extern "C" int qlora_binding_layouts(const void* table, void* const* objects, int64_t n,
                                     int64_t* at, int64_t* layout) {
  const Table* t = static_cast<const Table*>(table);
  if (n == 0) return t->major == 1 && t->view ? 0 : -1;
  for (int64_t i = 0; i < n; ++i) {
    View v;
    if (t->view(objects[i], &v)) return -1;
    at[i] = (int64_t)((uintptr_t)v.data + v.byte_offset);
    int64_t* l = layout + 6 * i;
    l[0] = (int64_t)v.code << 32 | v.bits << 16 | v.lanes;
    l[1] = (int64_t)v.device_type << 32 | (uint32_t)v.device_id;
    for (int k = 0; k < 2; ++k) {
      l[2 + k] = v.ndim == 2 ? v.shape[k] : -1;
      l[4 + k] = v.ndim == 2 ? v.strides[k] : -1;
    }
    if (l[2] <= 1 || l[3] == 0) l[4] = 0;   // of no meaning, and whatever it was given
    if (l[3] <= 1 || l[2] == 0) l[5] = 0;
  }
  return 0;
}
