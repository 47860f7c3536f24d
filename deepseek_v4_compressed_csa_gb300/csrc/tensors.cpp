// What checks.c asks of a tensor (type, device, layout, shape, address), from the tensor itself: 0.02 us a tensor, where
// asking by its Python attributes takes 0.3.  An own library, without which the checks ask by attributes: it needs torch's
// headers, which lay a tensor's members out in it, so it is of use to the torch that it was built for alone.
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

// That torch: its version and commit (CSA_TORCH, from the build).
extern "C" const char* csa_tensors_torch(void) { return CSA_TORCH; }

// 1: a dense CUDA tensor of this dtype and at most max_dims dimensions, its shape in dims[0 .. n); 0: another tensor;
// -1: no plain tensor (a subclass may answer for itself).
extern "C" int csa_tensor(PyObject* o, PyObject* dtype, int max_dims, int* n, long long* dims, long long* dev, void** p) {
  if (!THPVariable_CheckExact(o) || !THPDtype_Check(dtype)) return -1;
  try {  // (a tensor without storage throws)
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.scalar_type() != reinterpret_cast<THPDtype*>(dtype)->scalar_type || t.dim() > max_dims ||
        !t.is_contiguous())
      return 0;
    *n = (int)t.dim();
    for (int i = 0; i < *n; ++i) dims[i] = t.size(i);
    *dev = t.get_device();
    *p = t.data_ptr();
    return 1;
  } catch (...) {
    return 0;
  }
}
